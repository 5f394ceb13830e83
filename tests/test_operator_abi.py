"""wan_rmsnorm and wan_linear refuse bad calls on the host, before any launch
(no GPU is touched: every call here returns before a CUDA call is made)."""
import ctypes

import pytest
import torch

from video_diffusion_transformer_fwd_b200 import build_lib, wan

EINVAL, EALIGN, EUNSUP, OK = wan.WAN_EINVAL, wan.WAN_EALIGN, wan.WAN_EUNSUPPORTED, wan.WAN_OK
MB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_lib.build(verbose=False)
    return wan.load()


def norm(**kw):
    a = dict(rows=4, D=64, x=1 * MB, x_dtype=wan.WAN_BF16, ldx=64, residual=2 * MB, res_dtype=wan.WAN_F32, ldr=64,
             gain=3 * MB, eps=1e-6, h_out=4 * MB, ldh=64, y=5 * MB, y_dtype=wan.WAN_FP8, ldy=64, row_scale=6 * MB,
             stream=None)
    a.update(kw)
    stream = a.pop("stream")
    return wan.wan_rmsnorm(wan.wan_rmsnorm_args(**a), stream)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), EINVAL), (dict(D=0), EINVAL), (dict(D=16385), EUNSUP), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL), (dict(x=None), EINVAL), (dict(y=None), EINVAL), (dict(row_scale=None), EINVAL),
    (dict(x_dtype=wan.WAN_FP8), EUNSUP), (dict(res_dtype=wan.WAN_FP8), EUNSUP), (dict(y_dtype=wan.WAN_FP8_ATTN), EUNSUP),
    (dict(x_dtype=9), EUNSUP), (dict(residual=None), EINVAL),            # h_out without a residual
    (dict(ldx=63), EINVAL), (dict(ldr=63), EINVAL), (dict(ldh=63), EINVAL), (dict(ldy=63), EINVAL),
    (dict(ldx=-64), EINVAL), (dict(ldx=1 << 62), EINVAL),
    (dict(x=MB + 2), EALIGN), (dict(residual=2 * MB + 4), EALIGN), (dict(gain=3 * MB + 4), EALIGN),
    (dict(h_out=4 * MB + 8), EALIGN), (dict(y=5 * MB + 1), EALIGN), (dict(row_scale=6 * MB + 2), EALIGN),
    (dict(y=MB), EINVAL),                                                # codes over bf16 x
    (dict(y=2 * MB + 16), EINVAL), (dict(h_out=2 * MB + 16), EINVAL),    # partial overlap with the residual
    (dict(h_out=2 * MB, ldh=72), EINVAL),                                # another stride than the residual it covers
    (dict(h_out=5 * MB), EINVAL),                                        # two outputs in one place
    (dict(row_scale=5 * MB + 16), EINVAL), (dict(y=3 * MB), EINVAL),     # over the gain
    # slices of one buffer that reach into each other's columns, directly or around the end of a row
    (dict(x=MB, ldx=128, y=MB + 112, ldy=256), EINVAL), (dict(x=MB, ldx=128, y=MB + 208, ldy=256), EINVAL),
    (dict(x=MB, ldx=128, y=MB + 128, ldy=128), EINVAL),                  # beside it, but another stride
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None), OK),
])
def test_rmsnorm_refusals(kw, code):
    assert norm(**kw) == code
    assert code == OK or wan.last_error()


def lin(**kw):
    a = dict(M=4, N=48, K=64, dtype=wan.WAN_FP8, a=1 * MB, lda=64, a_scale=2 * MB, w=3 * MB, ldw=64, w_scale=4 * MB,
             w_scale_rows=1, bias=5 * MB, activation=wan.WAN_ACT_SILU, residual=6 * MB, res_dtype=wan.WAN_F32, ldr=48,
             out=7 * MB, out_dtype=wan.WAN_F32, ldo=48, stream=None)
    a.update(kw)
    stream = a.pop("stream")
    return wan.wan_linear(wan.wan_linear_args(**a), stream)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), EINVAL), (dict(N=-1), EINVAL), (dict(K=0), EINVAL), (dict(K=-8), EINVAL),
    (dict(dtype=wan.WAN_F32), EUNSUP), (dict(dtype=wan.WAN_FP8_ATTN), EUNSUP), (dict(out_dtype=wan.WAN_FP8), EUNSUP),
    (dict(res_dtype=7), EUNSUP), (dict(activation=4), EUNSUP), (dict(activation=-1), EUNSUP), (dict(w_scale_rows=2), EINVAL),
    (dict(a=None), EINVAL), (dict(w=None), EINVAL), (dict(out=None), EINVAL), (dict(a_scale=None), EINVAL),
    (dict(w_scale=None), EINVAL), (dict(lda=72), EALIGN), (dict(ldw=72), EALIGN),
    (dict(dtype=wan.WAN_BF16, lda=68), EALIGN), (dict(dtype=wan.WAN_BF16, ldw=68), EALIGN),
    (dict(lda=48), EINVAL), (dict(ldw=48), EINVAL), (dict(ldr=47), EINVAL), (dict(ldo=47), EINVAL),
    (dict(a=MB + 8), EALIGN), (dict(w=3 * MB + 8), EALIGN), (dict(bias=5 * MB + 2), EALIGN), (dict(out=7 * MB + 4), EALIGN),
    (dict(a_scale=2 * MB + 2), EALIGN), (dict(w_scale=4 * MB + 4), EALIGN),
    (dict(w_scale=4 * MB + 2, w_scale_rows=0), EALIGN), (dict(residual=6 * MB + 4), EALIGN),
    (dict(out=1 * MB), EINVAL), (dict(out=3 * MB), EINVAL), (dict(out=5 * MB), EINVAL), (dict(out=4 * MB), EINVAL),
    (dict(out=6 * MB + 16), EINVAL), (dict(out=6 * MB, ldo=64), EINVAL),
    (dict(out=6 * MB, out_dtype=wan.WAN_BF16), EINVAL),                  # another type than the residual it covers
    (dict(N=(1 << 31) - 1), EINVAL),
    (dict(M=0), OK), (dict(N=0), OK),
])
def test_linear_refusals(kw, code):
    assert lin(**kw) == code
    assert code == OK or wan.last_error()


def test_null_arguments():
    assert wan.wan_rmsnorm(None, None) == EINVAL and wan.wan_linear(None, None) == EINVAL


def test_packed_layouts_are_the_structs():
    """The helpers' packed arguments have the layout of the ctypes structures."""
    for fmt, cls in ((wan._LINEAR_ARGS, wan.wan_linear_args), (wan._RMSNORM_ARGS, wan.wan_rmsnorm_args)):
        assert fmt.size == ctypes.sizeof(cls)
        values = list(range(1, len(cls._fields_) + 1))
        got = cls.from_buffer_copy(fmt.pack(*values))
        assert [getattr(got, n) for n, _ in cls._fields_] == values


def test_python_helpers_refuse_host_tensors():
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        wan.rmsnorm(x)
    with pytest.raises(ValueError):
        wan.linear(x.bfloat16(), torch.zeros(8, 64, dtype=torch.bfloat16))

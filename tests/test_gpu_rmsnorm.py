"""wan_rmsnorm on the GPU against the formula in 64 bits, element by element.

Bounds (u = 2^-24, half a step of float32): h is one addition (u |h|), then
its storage (half a step of its type). The sum of squares adds at most 32
terms in one thread and 10 across the CTA, each step off by u, and h^2 by 2 u
(from h): rstd, whose relative error is half of the sum's plus a division, an
addition, a root and a division, is off by (44 / 2 + 4) u; y adds h's u and
two products: 29 u in all, held to 32 u. The scale of the codes is one
division more; a code is off by half a step of e4m3, 2^-4 of the value and at
least 2^-10 (half of the subnormal step), of a value that is itself off by
32 u and the two roundings of its factor."""
import numpy as np
import pytest
import torch

from oracle import wan_oracle as O
from video_diffusion_transformer_fwd_b200 import wan

from parity_util import Guarded, np64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.uint8}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wan.load()


def make(rows, D, x="bf16", r="f32", seed=0, spread=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows * 131 + D)
    row = torch.exp2(torch.randint(-spread, spread + 1, (rows, 1), device="cuda", generator=g).float())
    xt = (torch.randn(rows, D, device="cuda", generator=g) * row).to(DT[x])
    rt = None if r is None else (2 * torch.randn(rows, D, device="cuda", generator=g) * row).to(DT[r])
    return xt, rt, 1 + 0.1 * torch.randn(D, device="cuda", generator=g)


def reference(x, r, g, eps=EPS):
    h = np64(x) + (0 if r is None else np64(r))
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h, y * (1 if g is None else np64(g))


def check(x, r, g, out, y, scale, h, eps=EPS):
    h64, y64 = reference(x, r, g, eps)
    if r is not None:
        half = HALF["bf16" if r.dtype == torch.bfloat16 else "f32"]
        assert (np.abs(np64(h) - h64) <= (U + half * (1 + U)) * np.abs(h64)).all()
    if out == "fp8":
        v, s = O.e4m3_decode(y.cpu().numpy()), np64(scale).reshape(y.shape[:-1] + (1,))
        s64 = np.abs(y64).max(-1, keepdims=True) / 448
        assert (np.abs(s - s64) <= 34 * U * s64).all()
        z = np.divide(y64, s64, out=np.zeros_like(y64), where=s64 > 0)
        assert (np.abs(v - z) <= np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10) * (1 + 2.0 ** -6) + 72 * U * np.abs(z)).all()
    else:
        assert (np.abs(np64(y) - y64) <= (32 * U + HALF[out] * (1 + 32 * U)) * np.abs(y64)).all()


# one thread to several per row, one warp, one CTA of every register depth; the
# same for widths that are not multiples of 8
WIDTHS = [8, 16, 64, 72, 128, 136, 256, 264, 512, 520, 1536, 2048, 2056, 4096, 5120, 8192, 8200, 13824, 16384]
RAGGED = [1, 3, 7, 9, 31, 33, 57, 58, 127, 129, 500, 507, 513, 603, 754, 755, 771, 1037, 2047, 2049, 7031, 16366, 16370, 16371, 16383]


@pytest.mark.parametrize("D", WIDTHS + RAGGED)
@pytest.mark.parametrize("out", ["bf16", "f32", "fp8"])
def test_widths(D, out):
    x, r, g = make(5, D)
    y, s, h = wan.rmsnorm(x, g, residual=r, out_dtype=out)
    check(x, r, g, out, y, s, h)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("r", [None, "bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("rows,D", [(1, 5120), (37, 128), (19, 1037), (300, 1536)])
def test_types(x, r, out, rows, D):
    xt, rt, g = make(rows, D, x, r, seed=3, spread=12)
    y, s, h = wan.rmsnorm(xt, g, residual=rt, out_dtype=out)
    check(xt, rt, g, out, y, s, h)
    assert (h is xt) == (r is None) and (s is None) == (out != "fp8")


@pytest.mark.parametrize("rows", [1, 2, 3, 7, 8, 9, 16, 17, 1000])
@pytest.mark.parametrize("D", [64, 71, 128, 200, 250, 1000, 1037])
def test_row_counts_and_guards(rows, D):
    """Rows that do not fill the last CTA; bytes around every output stay."""
    x, r, g = make(rows, D)
    gy, gs, gh = Guarded((rows, D), torch.uint8), Guarded((rows,), torch.float32), Guarded((rows, D), torch.float32)
    wan.rmsnorm(x, g, residual=r, out=gy.t, row_scale=gs.t, h_out=gh.t)
    for b in (gy, gs, gh):
        b.check()
    check(x, r, g, "fp8", gy.t, gs.t, gh.t)


@pytest.mark.parametrize("D", [96, 1536, 1037])
def test_codes_are_those_of_the_quantizer(D):
    """The e4m3 output is wan_quantize_fp8 of the float32 output, bit for bit."""
    x, r, g = make(64, D, seed=9, spread=10)
    y32, _, _ = wan.rmsnorm(x, g, residual=r, out_dtype="f32")
    q, s, _ = wan.rmsnorm(x, g, residual=r, out_dtype="fp8")
    if D % 4 == 0:
        q2, s2 = wan.quantize_fp8(y32)
        assert torch.equal(q, q2) and torch.equal(s, s2)
    else:
        qr, sr = O.quantize_fp8(np64(y32), per_row=True)
        assert np.array_equal(O.e4m3_decode(q.cpu().numpy()), qr) and np.array_equal(np64(s), sr[:, 0])


def test_no_gain_no_stored_sum_and_leading_axes():
    x, r, _ = make(6, 256)
    y, _, h = wan.rmsnorm(x.view(2, 3, 256), residual=r.view(2, 3, 256), out_dtype="f32")
    assert y.shape == h.shape == (2, 3, 256)
    check(x, r, None, "f32", y.view(6, 256), None, h.view(6, 256))
    y2 = torch.empty_like(y)
    args = wan.wan_rmsnorm_args(x=x.data_ptr(), residual=r.data_ptr(), y=y2.data_ptr(), ldx=256, ldr=256, ldy=256, rows=6,
                                D=256, x_dtype=wan.WAN_BF16, res_dtype=wan.WAN_F32, y_dtype=wan.WAN_F32, eps=EPS)
    assert wan.wan_rmsnorm(args, torch.cuda.current_stream().cuda_stream) == wan.WAN_OK
    torch.cuda.synchronize()
    assert torch.equal(y, y2)


# pads of x, residual, y, h_out: strides that agree modulo 8 (aligned rows, and
# shifted ones with widths that end anywhere), and strides that do not
@pytest.mark.parametrize("D,pads", [(256, (8, 8, 8, 8)), (256, (24, 8, 0, 16)), (250, (6, 6, 6, 6)), (250, (1, 9, 1, 17)),
                                    (1003, (2, 2, 10, 2)), (1000, (5, 5, 5, 5)), (1000, (5, 6, 7, 9)), (256, (1, 2, 3, 4)),
                                    (5, (3, 4, 0, 1)), (3001, (0, 1, 2, 0)), (9000, (1, 0, 0, 0))])
def test_strided_rows_leave_the_gaps(D, pads):
    """Rows further apart than D: NaN between input rows is not read, and what
    lies between output rows stays."""
    rows = 9
    x, r, g = make(rows, D)
    big = [torch.full((rows, D + p), float("nan"), device="cuda", dtype=t.dtype) for t, p in zip((x, r), pads)]
    for b, t in zip(big, (x, r)):
        b[:, :D] = t
    outs = [torch.full((rows, D + p), 7, device="cuda", dtype=torch.float32) for p in pads[2:]]
    y, _, h = wan.rmsnorm(big[0][:, :D], g, residual=big[1][:, :D], out=outs[0][:, :D], h_out=outs[1][:, :D])
    check(x, r, g, "f32", y, None, h)
    assert all(bool((o[:, D:] == 7).all()) for o in outs)
    y1, _, h1 = wan.rmsnorm(x, g, residual=r, out_dtype="f32")
    assert torch.allclose(y1, y, rtol=64 * U, atol=0) and torch.equal(h1, h)


def test_in_place():
    for D in (512, 1037, 3163):
        x, r, g = make(11, D, r="bf16")
        y, _, h = wan.rmsnorm(x, g, residual=r)
        x2, r2 = x.clone(), r.clone()
        wan.rmsnorm(x2, g, residual=r2, out=x2, h_out=r2)
        assert torch.equal(x2, y) and torch.equal(r2, h)


def test_zero_infinite_and_nan_rows():
    x, r, g = make(6, 512, x="f32")
    x[1], r[1] = 0, 0
    x[2, 5], x[3, 7] = float("nan"), float("inf")
    x[4] *= 1e-30; r[4] *= 1e-30
    for out in ("f32", "bf16"):
        y, _, h = wan.rmsnorm(x, g, residual=r, out_dtype=out)
        assert not y[1].any() and y[2].isnan().all() and y[3, 7].isnan() and not y[3, :7].any()
        keep = [0, 1, 4, 5]
        check(x[keep], r[keep], g, out, y[keep], None, h[keep])
    q, s, _ = wan.rmsnorm(x, g, residual=r, out_dtype="fp8")
    assert not q[1].any() and s[1] == 0 and s[2].isnan() and s[3].isnan()
    assert bool(((q[2] & 127) == 127).all())
    keep = [0, 4, 5]
    y64 = reference(x[keep], r[keep], g)[1]
    deq = O.e4m3_decode(q[keep].cpu().numpy()) * np64(s[keep])[:, None]
    assert (np.abs(deq - y64) <= 2.0 ** -4 * 1.02 * np.abs(y64) + 2.0 ** -9 * np64(s[keep])[:, None]).all()
    y0, _, _ = wan.rmsnorm(x[1:2], g, residual=r[1:2], eps=0.0, out_dtype="f32")
    assert y0.isnan().all()                                    # 0 / 0, as the formula says


def test_empty_call():
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    y, s, h = wan.rmsnorm(x, out_dtype="fp8")
    assert y.shape == (0, 64) and s.shape == (0,) and h is x


def test_long_rows_pass_32_bits():
    """More than 2^31 elements: the last rows land where they belong."""
    rows, D = 262160, 8208
    x = torch.zeros(rows, D, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(5)
    last = torch.randn(3, D, device="cuda", generator=g).bfloat16()
    x[-3:] = last
    y = torch.full((rows, D), 9, device="cuda", dtype=torch.uint8)
    _, s, _ = wan.rmsnorm(x, out=y)
    check(last, None, None, "fp8", y[-3:], s[-3:], None)
    assert not y[:-3].any() and not s[:-3].any()


def test_streams_and_a_captured_graph():
    x, r, g = make(40, 1536)
    want, ws, wh = wan.rmsnorm(x, g, residual=r, out_dtype="fp8")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q, s, h = wan.rmsnorm(x, g, residual=r, out_dtype="fp8", stream=side)
    side.synchronize()
    assert torch.equal(q, want) and torch.equal(s, ws) and torch.equal(h, wh)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, s, h = wan.rmsnorm(x, g, residual=r, out_dtype="fp8")
    x2, r2, _ = make(40, 1536, seed=77)
    x.copy_(x2); r.copy_(r2)
    graph.replay()
    want, ws, wh = wan.rmsnorm(x2, g, residual=r2, out_dtype="fp8")
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(s, ws) and torch.equal(h, wh)


def test_python_refusals():
    x, r, g = make(4, 64)
    for kw in (dict(gain=g[:32]), dict(gain=g.bfloat16()), dict(residual=r[:3]), dict(residual=r.half()),
               dict(h_out=r.clone()), dict(out=r, out_dtype="bf16"), dict(row_scale=g[:4]), dict(residual=r.cpu()),
               dict(out=torch.empty(4, 65, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            wan.rmsnorm(x, **kw)
    with pytest.raises(ValueError):
        wan.rmsnorm(torch.empty(64, 4, device="cuda", dtype=torch.bfloat16).t())
    with pytest.raises(wan.WanError):
        wan.rmsnorm(x[:1].expand(4, 64))                       # rows on top of one another
    with pytest.raises(wan.WanError):
        wan.rmsnorm(torch.empty(2, 16392, device="cuda"))

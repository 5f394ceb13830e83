"""wan_rmsnorm on rows whose strides do not agree, which pass through shared
memory: amounts around what a kernel gets unasked (48 KB), and calls of several
host threads at once."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from video_diffusion_transformer_fwd_b200 import wan

from test_gpu_rmsnorm import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wan.load()


@pytest.mark.parametrize("x,r,D", [("f32", None, D) for D in (12200, 12216, 12224, 12248, 12276, 12280, 12284)] +
                         [("bf16", "f32", D) for D in (6104, 6109, 6112, 6121, 6136, 6140)])
def test_widths_around_48_kb(x, r, D):
    """Rows of 12224 float32, or of 6112 twice, with 16 bytes each to align them,
    take 48 KB less what the kernel holds by itself."""
    xt, rt, g = make(3, D, x, r, seed=D)
    wide = torch.zeros(3, D + 1, device="cuda", dtype=xt.dtype)
    wide[:, :D] = xt
    y = torch.empty(3, (D + 7) // 8 * 8, device="cuda")[:, :D] if D % 8 else torch.empty(3, D, device="cuda")
    y, s, h = wan.rmsnorm(wide[:, :D], g, residual=rt, out=y)
    check(xt, rt, g, "f32", y, s, h)


@pytest.mark.parametrize("out", ["f32", "fp8"])
def test_threads_with_rows_of_different_widths(out):
    """Rows whose strides do not agree, of widths that need different amounts of
    shared memory in the same kernel (131, 104 and 72 KB), from three threads."""
    calls = []
    for D in (16384, 13000, 9000):
        x, r, g = make(3, D, "f32", "f32", seed=D)
        wide = torch.zeros(3, D + 1, device="cuda")
        wide[:, :D] = x
        calls.append((wide[:, :D], r, g, wan.rmsnorm(wide[:, :D], g, residual=r, out_dtype=out)))
        check(x, r, g, out, *calls[-1][3])
    torch.cuda.synchronize()

    def many(call):
        x, r, g, (y, s, h) = call
        st = torch.cuda.Stream()
        got = [torch.empty_like(t) if t is not None else None for t in (y, s, h)]
        for _ in range(2000):
            wan.rmsnorm(x, g, residual=r, out=got[0], row_scale=got[1], h_out=got[2], stream=st)
        st.synchronize()
        return got

    with ThreadPoolExecutor(3) as pool:
        got = list(pool.map(many, calls))
    for (_, _, _, want), out3 in zip(calls, got):
        assert all(torch.equal(a, b) for a, b in zip(want, out3) if a is not None)
    assert wan.device_status() == wan.WAN_OK


@pytest.mark.parametrize("D,pad", [(128, 0), (1003, 0), (1000, 5), (5120, 0), (9000, 1)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_rows_do_not_reach_each_other(D, pad, poison):
    """Every third row of a call, when the other rows of x and of the residual
    turn into NaN or infinities: the same bits (aligned rows, rows off a boundary
    and rows whose strides do not agree)."""
    x, r, g = make(31, D)
    wide = torch.zeros(31, D + pad, device="cuda", dtype=x.dtype)
    wide[:, :D] = x
    for out in ("bf16", "f32", "fp8"):
        before = wan.rmsnorm(wide[:, :D], g, residual=r, out_dtype=out)
        x2, r2 = wide.clone(), r.clone()
        others = torch.ones(31, device="cuda", dtype=torch.bool)
        others[::3] = False
        x2[others], r2[others] = poison, poison
        after = wan.rmsnorm(x2[:, :D], g, residual=r2, out_dtype=out)
        for a, b in zip(before, after):
            assert a is None or torch.equal(a[::3], b[::3])


def test_captured_before_any_call_at_these_widths():
    """Kernels that no call has launched yet, captured: rows of every layout."""
    xs = [make(5, D, "f32", "bf16", seed=D) for D in (24, 90, 200, 450, 700, 2100, 8500)]
    wide = torch.randn(5, 5001, device="cuda")
    outs = []
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, r, g in xs:
            outs.append(wan.rmsnorm(x, g, residual=r, out_dtype="bf16"))
        outs.append(wan.rmsnorm(wide[:, :5000], None, out=torch.empty(5, 5000, device="cuda")))
    graph.replay()
    torch.cuda.synchronize()
    for (x, r, g), (y, s, h) in zip(xs, outs):
        check(x, r, g, "bf16", y, s, h)
    check(wide[:, :5000], None, None, "f32", *outs[-1])

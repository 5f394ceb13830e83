"""wan_linear under calls that its documentation allows beside the plain one:
after other calls of the same sizes, from several threads, on rows more than
2^31 elements apart, captured at sizes that never ran, and on a device where an
earlier wait gave up."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from video_diffusion_transformer_fwd_b200 import wan

from test_gpu_linear import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wan.load()


def new_thread(call):
    """call() on a thread that has made no call before."""
    with ThreadPoolExecutor(1) as pool:
        return pool.submit(call).result()


@pytest.mark.parametrize("M", [5, 2500])
def test_first_call_of_a_thread(M):
    """A thread that has made no CUDA call of its own."""
    c = Case(M, 512, 256, f8=True, res="f32", out="f32")
    out = torch.empty_like(c.r)
    want = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.current_stream()
    new_thread(lambda: c.run(out=out, stream=s))
    torch.cuda.synchronize()
    assert torch.equal(out, want)


# float32 outputs show every change in the order of a sum
@pytest.mark.parametrize("M,N,K", [(20, 700, 4096), (100, 1000, 2048), (100, 1500, 4096), (150, 900, 3000), (260, 1100, 1536),
                                   (300, 640, 2560), (600, 512, 4096), (1100, 320, 5120), (1500, 512, 2048)])
@pytest.mark.parametrize("f8", [False, True])
def test_results_do_not_depend_on_the_calls_before(M, N, K, f8):
    K = K // 16 * 16
    c = Case(M, N, K, f8, res="f32", out="f32")

    def both(*residuals):
        return [c.run(residual=r) for r in residuals]

    first, second = new_thread(lambda: both(c.r, None)), new_thread(lambda: both(None, c.r))
    torch.cuda.synchronize()
    assert torch.equal(first[0], second[1]) and torch.equal(first[1], second[0])


def test_four_threads_at_once():
    cs = [Case(M, N, K, f8, "gelu_tanh", res="bf16", out="bf16", seed=M)
          for M, N, K, f8 in ((1, 1536, 4096, False), (24, 2000, 1024, True), (300, 1003, 1000, False), (2500, 512, 768, True))]
    want = [c.run() for c in cs]
    torch.cuda.synchronize()

    def many(c):
        st = torch.cuda.Stream()
        outs = [torch.empty_like(c.r) for _ in range(30)]
        for o in outs:
            c.run(out=o, stream=st)
        st.synchronize()
        return outs

    with ThreadPoolExecutor(4) as pool:
        got = list(pool.map(many, cs))
    assert all(torch.equal(o, w) for outs, w in zip(got, want) for o in outs)


@pytest.mark.parametrize("M,N,ld", [(40, 200, 1 << 26), (40, 203, (1 << 26) + 3), (2304, 264, 1 << 20)])
def test_rows_pass_32_bits(M, N, ld):
    """Few rows and CTA pairs, an output and a residual in place whose last rows
    lie more than 2^31 elements behind the first."""
    c = Case(M, N, 256, res="bf16")
    flat = torch.zeros((M - 1) * ld + N, device="cuda", dtype=torch.bfloat16)
    out = flat.as_strided((M, N), (ld, 1))
    out.copy_(c.r)
    assert out.stride(0) * (M - 1) > 2 ** 31
    c.run(residual=out, out=out)
    c.check(out.contiguous())
    assert int(flat.count_nonzero()) <= M * N
    assert wan.device_status() == wan.WAN_OK


def test_capture_at_new_sizes():
    """Sizes that no call had before the capture."""
    cs = [Case(M, N, K, f8, "silu", res="f32", out="f32") for M, N, K, f8 in
          ((3, 1111, 2056, False), (77, 1311, 2064, True), (1111, 515, 528, False), (3333, 777, 1040, True))]
    outs = [torch.zeros(c.r.shape, device="cuda") for c in cs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, o in zip(cs, outs):
            c.run(out=o)
    graph.replay()
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        c.check(o)


@pytest.mark.parametrize("M,N,K,f8", [(1, 1536, 8192, False), (37, 600, 8192, True), (90, 520, 6400, False), (2304, 512, 640, True)])
def test_after_a_wait_that_gave_up(M, N, K, f8):
    """Launches on a device whose status is set end at once, the context stays
    usable, and the same call is right once the status has been read."""
    s = torch.cuda.current_stream().cuda_stream
    c = Case(M, N, K, f8, res="f32", out="f32")
    wan.check(wan.wan_selftest_watchdog(s))
    for _ in range(3):
        c.run()
    assert wan.wan_device_status(s) == wan.WAN_ETIMEOUT
    assert wan.wan_device_status(s) == wan.WAN_OK
    c.check(c.run())
    assert wan.device_status() == wan.WAN_OK


@pytest.mark.parametrize("rows", [1, 6, 700])
@pytest.mark.parametrize("D", [128, 136])
def test_slices_of_one_buffer(rows, D):
    """Inputs and outputs side by side in the rows of a packed buffer, and scales
    that begin at any row."""
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    buf = torch.randn(rows, 3 * D + 40, device="cuda", generator=g).bfloat16()
    w = torch.randn(D, D, device="cuda", generator=g).bfloat16()
    before = buf.clone()
    a, y, out, rest = buf[:, :D], buf[:, D:2 * D], buf[:, 2 * D:3 * D], buf[:, 3 * D:]
    want, _, _ = wan.rmsnorm(a.clone())
    wan.rmsnorm(a, out=y)
    assert torch.equal(y, want)
    wan.linear(y, w, residual=a, out=out)
    assert torch.equal(out, wan.linear(want, w, residual=before[:, :D].contiguous()))
    assert torch.equal(a, before[:, :D]) and torch.equal(rest, before[:, 3 * D:])
    if rows > 5 and D % 16 == 0:
        q, s = wan.quantize_fp8(want)
        wq, ws = wan.quantize_fp8(w, per_row=False)
        full = wan.linear(q, wq, a_scale=s, w_scale=ws)
        part = wan.linear(q[3:], wq, a_scale=s[3:], w_scale=ws)
        assert float((part.float() - full[3:].float()).norm()) <= 2.0 ** -8 * float(full.float().norm())
        scales = torch.zeros(rows, device="cuda")
        wan.rmsnorm(want[:rows - 1].contiguous(), out_dtype="fp8", row_scale=scales[1:])
        assert scales[0] == 0 and (scales[1:] > 0).all()


@pytest.mark.parametrize("M,N", [(5984, 155), (5000, 153), (5000, 158), (4000, 1001), (2600, 2559), (64, 155)])
@pytest.mark.parametrize("res", [None, "bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_rows_that_end_inside_16_bytes(M, N, res, out):
    """Rows that begin on 16-byte boundaries and end inside one: what lies behind
    them stays, with a residual of its own and with one in place."""
    c = Case(M, N, 520, act="relu", res=res, out=out)
    ld = (N + 7) // 8 * 8
    full = torch.full((M, ld), 7.0, device="cuda", dtype=c.out)
    o = full[:, :N]
    kw = {}
    if res == out:
        o.copy_(c.r)
        kw = dict(residual=o)
    c.run(out=o, **kw)
    assert (full[:, N:] == 7).all()
    c.check(o, list(range(0, M, max(1, M // 100))))
    assert wan.device_status() == wan.WAN_OK


@pytest.mark.parametrize("M,N,K,f8", [(24, 13424, 2064, False), (32, 12072, 1552, False), (20, 12000, 4096, False),
                                      (26, 12808, 4112, True), (29, 13504, 3000, False)])
def test_few_tokens_three_ctas_to_an_sm(M, N, K, f8):
    """17 to 32 tokens of so many weight rows that three CTAs share an SM and the
    sums meet in the ring's memory; one call after another on a stream."""
    c = Case(M, N, K, f8, "silu", res="bf16", out="f32")
    first = c.run()
    outs = [c.run() for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
    c.check(first)
    assert wan.device_status() == wan.WAN_OK


@pytest.mark.parametrize("M,N,K", [(7, 1500, 4096), (24, 640, 5120), (48, 640, 5120), (333, 1003, 1000), (2304, 512, 640), (3000, 155, 2560)])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), 1e30])
def test_rows_do_not_reach_each_other(M, N, K, f8, poison):
    """Every third row of a call, when the other rows of a, of its scales and of
    the residual turn into NaN, infinities or large values: the same bits."""
    K = K // 16 * 16 if f8 else K
    c = Case(M, N, K, f8, "silu", res="f32", out="f32")
    before = c.run()
    keep = torch.arange(0, M, 3, device="cuda")
    others = torch.ones(M, device="cuda", dtype=torch.bool)
    others[keep] = False
    if f8:
        c.a[others] = 127 if poison != 1e30 else 126            # NaN, or the largest code
        c.sa[others] = poison
    else:
        c.a[others] = poison
    c.r[others] = poison
    after = c.run()
    torch.cuda.synchronize()
    assert torch.equal(before[keep], after[keep]) and torch.isfinite(after[keep]).all()
    assert not torch.equal(before[others], after[others])
    assert wan.device_status() == wan.WAN_OK


@pytest.mark.parametrize("M,N,K", [(1, 1024, 13824), (24, 520, 13824), (100, 384, 8192), (300, 640, 2048), (2304, 1003, 2048), (2500, 512, 13824)])
def test_float32_output_loses_no_more_than_a_part(M, N, K):
    """The tensor core's rounding toward zero counts 1.1e-9 for each element of K
    of a part, and a part has 2048 at most: 2.3e-6 of the product's norm, and the
    float32 additions of its parts (14 at most, 2^-24 each)."""
    c = Case(M, N, K, bias=False, out="f32")
    want = c.a.double() @ c.w.double().t()
    err = float((c.run().double() - want).norm() / want.norm())
    assert err <= 2.3e-6 + 14 * 2.0 ** -24, err

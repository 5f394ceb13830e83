"""wan_rmsnorm and wan_linear one after another: every call may start before the
one in front of it on the stream has ended, so long dependent chains, chains
through the library's other kernels and through torch's, captured and not,
have to give what the same calls give one at a time."""
import pytest
import torch

from video_diffusion_transformer_fwd_b200 import wan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wan.load()


class Chain:
    """`depth` pre-norm sublayers on one float32 stream, buffers reused from
    layer to layer, so that a call that starts too early reads or overwrites
    what the one before still uses."""

    def __init__(self, rows, D, F, depth, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        self.x0, self.D, self.F, self.rows = rnd(rows, D), D, F, rows
        self.gain = [1 + 0.1 * rnd(D) for _ in range(depth)]
        self.w1 = [wan.quantize_fp8((rnd(F, D) * D ** -0.5).bfloat16()) for _ in range(depth)]
        self.w2 = [(rnd(D, F) * F ** -0.5).bfloat16() for _ in range(depth)]
        self.b1 = [0.1 * rnd(F).bfloat16() for _ in range(depth)]
        self.x, self.x2 = self.x0.clone(), torch.empty(rows, D, device="cuda")
        self.branch = torch.zeros(rows, D, device="cuda", dtype=torch.bfloat16)
        self.q, self.qs = torch.empty(rows, D, device="cuda", dtype=torch.uint8), torch.empty(rows, device="cuda")
        self.u = torch.empty(rows, F, device="cuda", dtype=torch.bfloat16)

    def run(self, between=lambda: None):
        self.x.copy_(self.x0)
        self.branch.zero_()
        a, b = self.x, self.x2
        for g, (w1, s1), w2, b1 in zip(self.gain, self.w1, self.w2, self.b1):
            wan.rmsnorm(self.branch, g, residual=a, out=self.q, row_scale=self.qs, h_out=b)
            between()
            wan.linear(self.q, w1, b1, "gelu_tanh", a_scale=self.qs, w_scale=s1, out=self.u)
            between()
            wan.linear(self.u, w2, out=self.branch)
            between()
            a, b = b, a
        wan.linear(self.u, self.w2[0], residual=a, out=a)
        between()
        return a


# one token and a ragged handful (K split over clusters), many rows (CTA pairs), an odd width
SHAPES = [(1, 1536, 4096), (37, 528, 1000), (700, 256, 1536), (2500, 512, 1024)]


@pytest.mark.parametrize("rows,D,F", SHAPES)
def test_long_chain_equals_one_call_at_a_time(rows, D, F):
    c = Chain(rows, D, F, 12, seed=rows)
    want = c.run(torch.cuda.synchronize).clone()
    torch.cuda.synchronize()
    for _ in range(10):
        got = c.run()
    assert torch.equal(got, want)
    assert wan.device_status() == wan.WAN_OK


@pytest.mark.parametrize("rows,D,F", SHAPES)
def test_captured_chain(rows, D, F):
    c = Chain(rows, D, F, 6, seed=rows + 1)
    want = c.run(torch.cuda.synchronize).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.run()
    for _ in range(5):
        c.x.fill_(float("nan"))
        c.x2.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_chains_on_two_streams_share_weights():
    a, b = Chain(5, 1536, 4096, 6, seed=3), Chain(400, 256, 1536, 6, seed=4)
    want = [c.run(torch.cuda.synchronize).clone() for c in (a, b)]
    torch.cuda.synchronize()
    sts = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for c, st in zip((a, b), sts):
            with torch.cuda.stream(st):
                got.append(c.run())
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_between_other_kernels_and_copies():
    """A torch kernel, a device copy, a memset and the library's own quantizer
    directly before and behind."""
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    rows, D = 300, 1024
    w, ws = wan.quantize_fp8((rnd(768, D) * 0.03).bfloat16())
    src = [rnd(rows, D).bfloat16() for _ in range(4)]
    big = torch.empty(64 << 20, device="cuda", dtype=torch.uint8)

    def once(x, buf, sync):
        buf.zero_()
        sync()
        buf.copy_(x)
        sync()
        buf.mul_(2)
        sync()
        y, _, _ = wan.rmsnorm(buf, out_dtype="bf16")
        sync()
        buf.zero_()                             # the norm has read it
        q, s = wan.quantize_fp8(y)
        sync()
        o = wan.linear(q, w, a_scale=s, w_scale=ws, activation="silu", out_dtype="f32")
        sync()
        q.zero_()                               # the product has read it
        big.zero_()
        return o * 2

    buf = torch.empty_like(src[0])
    want = [once(x, buf, torch.cuda.synchronize) for x in src]
    for _ in range(20):
        got = [once(x, buf, lambda: None) for x in src]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))

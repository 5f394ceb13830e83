"""wan_linear on the GPU against the formula in 64 bits, element by element.

Bounds: sums of K exact products in float32 are off by at most
(K + 8) 2^-24 sum |a w| (the bound of wan_linear_fp8's test). The activations
are z / (1 + exp(-u)) with |derivative| <= 1.13, exp off by
(2 + 1.173 |u|) 2^-23 and its argument by |u| 2^-22, the division by 2^-22:
(6 + 3.2 |u|) 2^-23 of the result, and at most 1e-36 where exp overflows. Then
the residual's addition (2^-24) and the output's half step."""
import numpy as np
import pytest
import torch

from oracle import wan_oracle as O
from video_diffusion_transformer_fwd_b200 import wan

from parity_util import Guarded, np64, rel_l2

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wan.load()


class Case:
    def __init__(self, M, N, K, f8=False, act="none", bias=True, res=None, out="bf16", rows_scale=True, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 7 * M + 11 * N + 13 * K)
        a = torch.randn(M, K, device="cuda", generator=g)
        w = torch.randn(N, K, device="cuda", generator=g) * K ** -0.5 * 2
        self.sa = self.sw = None
        if f8:
            self.sa = a.abs().amax(1) / 448
            self.sw = w.abs().amax(1) / 448 if rows_scale else w.abs().amax().reshape(1) / 448
            self.a = (a / self.sa[:, None]).to(F8).view(torch.uint8)
            self.w = (w / self.sw[:, None]).to(F8).view(torch.uint8)
        else:
            self.a, self.w = a.bfloat16(), w.bfloat16()
        self.b = torch.randn(N, device="cuda", generator=g).bfloat16() if bias else None
        self.r = None if res is None else torch.randn(M, N, device="cuda", generator=g).to(DT[res])
        self.act, self.out, self.f8 = act, DT[out], f8

    def args(self):
        return dict(bias=self.b, activation=self.act, residual=self.r, a_scale=self.sa, w_scale=self.sw)

    def run(self, **kw):
        o = kw.pop("out", None)
        if o is None:
            o = torch.empty(self.a.shape[0], self.w.shape[0], device="cuda", dtype=self.out)
        return wan.linear(self.a, self.w, out=o, **{**self.args(), **kw})

    def operands(self, rows):
        dec = (lambda t: O.e4m3_decode(t.cpu().numpy())) if self.f8 else np64
        a, w = dec(self.a[rows]), dec(self.w)
        if self.f8:
            a, w = a * np64(self.sa[rows])[:, None], w * np64(self.sw)[:, None]
        return a, w

    def check(self, got, rows=None):
        if rows is None:
            rows = slice(None)
        else:
            assert min(rows) >= 0 and max(rows) < got.shape[0]
            rows = torch.as_tensor(rows, device="cuda")
        a, w = self.operands(rows)
        K = a.shape[1]
        z = a @ w.T + (0 if self.b is None else np64(self.b))
        mag = np.abs(a) @ np.abs(w).T + (0 if self.b is None else np.abs(np64(self.b)))
        ez = (K + 8) * 2.0 ** -24 * mag
        y, e = activated(z, self.act)
        e = e + 1.13 * ez
        if self.r is not None:
            y = y + np64(self.r[rows])
            e = e + 2.0 ** -24 * (np.abs(y) + e)
        err = np.abs(np64(got[rows]) - y)
        bound = e + HALF[got.dtype] * (np.abs(y) + e) + 1e-36
        assert (err <= bound).all(), float((err / bound).max())


def activated(z, act):
    """act(z) and the bound of its own error."""
    if act == "none":
        return z, 0.0
    if act == "relu":
        return np.maximum(z, 0), 0.0
    u = z if act == "silu" else 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
    with np.errstate(over="ignore"):
        y = z / (1 + np.exp(-u))
    return y, (6 + 3.2 * np.minimum(np.abs(u), 100)) * 2.0 ** -23 * np.abs(y)


# rows: one token, a full and a ragged group of 16, several tiles; columns and
# K that end inside a tile; K shorter than one step
SIZES = [(1, 1, 8), (1, 128, 64), (2, 5, 40), (3, 129, 72), (15, 64, 128), (16, 128, 128), (17, 1003, 1000),
         (33, 256, 4160), (130, 384, 640), (257, 136, 520), (300, 1000, 1536), (511, 77, 96)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("f8", [False, True])
def test_sizes(M, N, K, f8):
    K = K // 16 * 16 if f8 and K > 16 else (16 if f8 else K)
    c = Case(M, N, K, f8, "gelu_tanh", res="f32", out="f32")
    c.check(c.run())
    assert wan.device_status() == wan.WAN_OK


@pytest.mark.parametrize("f8,rows_scale", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("bias,res,out", [(True, "f32", "f32"), (False, "bf16", "bf16"), (True, None, "bf16"),
                                          (False, None, "f32"), (True, "f32", "bf16"), (True, "bf16", "f32")])
def test_types_and_activations(f8, rows_scale, act, bias, res, out):
    for M, N, K in ((1, 300, 256), (70, 203, 1024)):
        c = Case(M, N, K, f8, act, bias, res, out, rows_scale, seed=5)
        c.check(c.run())


@pytest.mark.parametrize("M,N,K,f8", [(1, 5120, 5120, False), (24, 13824, 5120, True), (512, 5120, 4096, False),
                                      (1000, 1536, 8960, True), (7800, 1536, 1536, False), (4100, 5120, 13824, True),
                                      (2500, 1029, 1536, False), (9000, 520, 5120, True)])
def test_workload_sizes(M, N, K, f8):
    c = Case(M, N, K, f8, "silu", res="bf16", out="bf16")
    got = c.run()
    assert wan.device_status() == wan.WAN_OK
    c.check(got, sorted({min(i, M - 1) for i in (0, 1, M // 3, M // 2, 2 * M // 3, max(M - 2, 0), M - 1)}))
    # every row against the library's own product (both rounded to bf16 or further)
    a, w = c.a.view(F8).float() if f8 else c.a.float(), c.w.view(F8).float() if f8 else c.w.float()
    z = a @ w.t()
    if f8:
        z = z * c.sa[:, None] * c.sw
    z = z + c.b.float()
    ref = z * torch.sigmoid(z) + c.r.float()
    assert float((got.float() - ref).norm() / ref.norm()) <= 2.0 ** -8


@pytest.mark.parametrize("M,N,K", [(16, 64, 16384), (300, 640, 9216), (1100, 320, 16384), (1, 256, 32768), (2300, 1300, 4104),
                                   (2300, 1031, 8200), (2048, 2048, 12296), (2500, 1100, 16384)])
def test_float32_output_of_long_bf16_sums(M, N, K):
    """A float32 output of bf16 operands keeps float32's worth: the tensor core
    rounds its running sum toward zero, at most 2^-23 a step of 16, so a chain
    of 256 steps (K = 4096) is off by 256 2^-23 / 2 = 1.5e-5 at the very most and
    by about a third of that on sums that grow along the way."""
    c = Case(M, N, K, bias=False, out="f32")
    a, w = c.operands(slice(None))
    assert rel_l2(np64(c.run()), a @ w.T) <= 1e-5


@pytest.mark.parametrize("M,N,K", [(1, 256, 8192), (2, 48, 70000), (120, 136, 40000), (500, 4000, 16384), (40, 512, 5120), (300, 640, 2048), (600, 1000, 4104), (2300, 1300, 768), (2300, 1300, 776),
                                   (2300, 1031, 8200), (5000, 1600, 1536), (9000, 520, 16384), (12000, 1111, 904)])
def test_float32_output_in_parts_of_k(M, N, K):
    """A running sum of at most 32 steps of 4 products, each rounded toward zero
    by at most 2^-23 of it and half of that in the mean, on sums that are two
    thirds of the last one: 128 / 2 * 2 / 3 * 2^-23 = 5e-6 with parts of 32
    steps, 2.5e-6 with the usual ones of at most 16."""
    c = Case(M, N, K, act="none", res="f32", out="f32")
    rows = torch.arange(0, M, max(1, M // 300), device="cuda")
    a, w = c.operands(rows)
    z = a @ w.T + np64(c.b)
    got = c.run()
    assert rel_l2(np64(got[rows]) - np64(c.r[rows]) - np64(c.b), z - np64(c.b)) <= (5e-6 if 1024 < K <= 2048 or K >= 16384 else 2.5e-6)
    c.check(got, rows.tolist())
    assert wan.device_status() == wan.WAN_OK


@pytest.mark.parametrize("M,N,K,f8", [(1, 136, 128, False), (5, 203, 256, True), (40, 1000, 200, False), (300, 129, 64, False),
                                      (2300, 264, 256, False), (2300, 133, 256, True)])
def test_strides_and_guards(M, N, K, f8):
    """Strided operands, residual and output; NaN between the rows of the
    operands is not read; bytes between and around the output's rows stay."""
    c = Case(M, N, K, f8, "silu", res="bf16", out="f32")
    want = c.run()
    pad = 32
    wide = lambda t, p: torch.nn.functional.pad(t.float() if t.dtype == torch.bfloat16 else t, (0, p), value=0x7F if t.dtype == torch.uint8 else float("nan")).to(t.dtype)  # noqa: E731
    a, w, r = wide(c.a, pad), wide(c.w, pad), wide(c.r, 3)
    go = Guarded((M, N + 5), torch.float32)
    go.t.fill_(7)
    wan.linear(a[:, :K], w[:, :K], out=go.t[:, :N], **{**c.args(), "residual": r[:, :N]})
    go.check()
    assert bool((go.t[:, N:] == 7).all())
    c.check(go.t[:, :N])
    assert torch.allclose(go.t[:, :N], want, rtol=1e-4, atol=1e-4)


@pytest.mark.parametrize("M,N", [(1, 128), (33, 200), (33, 203), (2300, 264), (2300, 263)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_residual_in_place(M, N, out):
    c = Case(M, N, 256, act="gelu_tanh", res=out, out=out)
    want = c.run()
    x = c.r.clone()
    c.run(residual=x, out=x)
    c.check(x)
    assert torch.equal(x, want)


def test_nan_and_infinities_stay_in_their_row():
    for M, N in ((5, 40), (2300, 264)):
        c = Case(M, N, 128, act="relu")
        want = c.run()
        c.a[2, 3] = float("nan")
        c.a[4, 0] = float("inf")
        got = c.run()
        assert got[2].isnan().all() and not torch.isfinite(got[4][c.w[:, 0] > 0]).any()
        keep = [i for i in range(M) if i not in (2, 4)]
        assert torch.equal(got[keep], want[keep])


def test_empty_calls_and_leading_axes():
    w = torch.randn(24, 64, device="cuda").bfloat16()
    assert wan.linear(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), w).shape == (0, 24)
    assert wan.linear(torch.zeros(3, 64, device="cuda", dtype=torch.bfloat16), w[:0]).shape == (3, 0)
    a = torch.randn(2, 3, 64, device="cuda").bfloat16()
    assert torch.equal(wan.linear(a, w), wan.linear(a.view(6, 64), w).view(2, 3, 24))


def test_deterministic_and_independent_of_the_other_rows():
    c = Case(48, 640, 5120, act="silu", out="f32")
    assert torch.equal(c.run(), c.run())


def test_streams_and_captured_graphs():
    """Two streams at once, and two captured graphs replayed at once, on calls
    that split K over a cluster."""
    cs = [Case(9, 1500, 4096, f8=f8, act="silu", seed=i) for i, f8 in ((1, False), (2, True))]
    want = [c.run() for c in cs]
    side = [torch.cuda.Stream() for _ in cs]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, st, o in zip(cs, side, outs):
            c.run(out=o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    for c, o in zip(cs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=o)
        graphs.append(g)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, side):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert wan.device_status() == wan.WAN_OK


def test_python_refusals():
    c = Case(4, 64, 64)
    f = Case(4, 64, 64, f8=True)
    for call in (lambda: c.run(a_scale=torch.ones(4, device="cuda")), lambda: f.run(a_scale=None),
                 lambda: f.run(w_scale=f.sw[:3]), lambda: c.run(bias=c.b.float()), lambda: c.run(bias=c.b[:8]),
                 lambda: c.run(residual=c.w[:4, :32]), lambda: wan.linear(c.a, f.w), lambda: wan.linear(c.a, c.w[:, :32]),
                 lambda: c.run(out=torch.empty(4, 64, device="cuda"), out_dtype="bf16"),
                 lambda: wan.linear(c.a, c.w.t()), lambda: wan.linear(c.a, c.w.cpu())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(KeyError):
        c.run(activation="tanh")
    with pytest.raises(wan.WanError):                          # rows that start on 2-byte boundaries
        wan.linear(torch.zeros(3, 65, device="cuda", dtype=torch.bfloat16), torch.zeros(8, 65, device="cuda", dtype=torch.bfloat16))


@pytest.mark.parametrize("rows", [1, 37, 700])
def test_pre_norm_sublayer(rows):
    """The operators as they are used together: norm with the residual's
    addition into codes, FP8 product with GELU, quantizer, FP8 product onto the
    stream; each stage against 64 bits on the inputs that it got."""
    D, Fh = 512, 1536
    g = torch.Generator(device="cuda").manual_seed(rows)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    branch, stream = rnd(rows, D).bfloat16(), 2 * rnd(rows, D)
    gain, b1, b2 = 1 + 0.1 * rnd(D), 0.1 * rnd(Fh).bfloat16(), 0.1 * rnd(D).bfloat16()
    w1, s1 = wan.quantize_fp8((0.05 * rnd(Fh, D)).bfloat16())
    w2, s2 = wan.quantize_fp8((0.05 * rnd(D, Fh)).bfloat16(), per_row=False)
    q, qs, h = wan.rmsnorm(branch, gain, residual=stream, out_dtype="fp8")
    u = wan.linear(q, w1, b1, "gelu_tanh", a_scale=qs, w_scale=s1)
    p, ps = wan.quantize_fp8(u)
    h0 = h.clone()
    wan.linear(p, w2, b2, residual=h, a_scale=ps, w_scale=s2, out=h)
    torch.cuda.synchronize()
    assert wan.device_status() == wan.WAN_OK
    first = Case(1, 1, 16, True, "gelu_tanh")
    first.a, first.w, first.sa, first.sw, first.b = q, w1, qs, s1, b1
    first.check(u)
    second = Case(1, 1, 16, True, "none", out="f32")
    second.a, second.w, second.sa, second.sw, second.b, second.r = p, w2, ps, s2, b2, h0
    second.check(h)
    # and the whole run against the sublayer without any rounding: three e4m3
    # roundings of relative size 2^-4 / sqrt(3) at most each on a branch that is
    # a part of the stream
    h64 = np64(branch) + np64(stream)
    y64 = h64 / np.sqrt((h64 ** 2).mean(-1, keepdims=True) + 1e-6) * np64(gain)
    dq = lambda t, s: O.e4m3_decode(t.cpu().numpy()) * (np64(s)[:, None])  # noqa: E731
    z = O.gelu_tanh(y64 @ dq(w1, s1).T + np64(b1))
    ref = z @ dq(w2, s2).T + np64(b2)
    assert rel_l2(np64(h) - h64, ref) <= 3 * 2.0 ** -4 / np.sqrt(3)

"""Kernels that share TMEM and shared memory of the SMs, from several host
threads at once, each on a stream of its own: wan_linear for few rows (clusters
whose CTAs wait for one another) and for many (CTA pairs), wan_rmsnorm, and the
two attentions, which take all of TMEM. Each result has the bits of the same
call alone."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from video_diffusion_transformer_fwd_b200 import wan

from test_gpu_linear import Case
from test_gpu_rmsnorm import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    wan.load()


def linear(sizes, f8):
    cases = [Case(M, N, K, f8, "silu", res="f32", out="f32", seed=i) for i, (M, N, K) in enumerate(sizes)]
    return [lambda st, c=c: (c.run(stream=st),) for c in cases]


def norms():
    rows = [make(*s) for s in ((1, 5120), (700, 1536), (50, 1037), (3000, 128))]
    return [lambda st, r=r: wan.rmsnorm(r[0], r[2], residual=r[1], out_dtype="fp8", stream=st) for r in rows]


def attentions(eight):
    g = torch.Generator(device="cuda").manual_seed(3)
    calls = []
    for B, L, H in ((1, 700, 4), (2, 300, 12), (1, 1500, 40)):
        q, k, v = (torch.randn(B, L, H, 128, device="cuda", generator=g).bfloat16() for _ in range(3))
        f = wan.attention_8bit if eight else wan.attention
        calls.append(lambda st, a=(q, k, v), f=f: (f(*a, stream=st),))
    return calls


def test_all_kernels_at_once():
    few = [(1, 5120, 4096), (20, 12000, 1024), (24, 3000, 5120), (90, 1024, 2048), (5, 200, 704)]
    many = [(2500, 512, 640), (1200, 2000, 1024)]
    work = [linear(few, False), linear([(M, N, K // 16 * 16) for M, N, K in few], True),
            linear(many, False) + norms(), attentions(False), attentions(True)]
    main = torch.cuda.current_stream()
    want = [[f(main) for f in calls] for calls in work]
    torch.cuda.synchronize()

    def run(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            got = [(j, work[i][j](st)) for _ in range(25) for j in range(len(work[i]))]
        st.synchronize()
        return all(torch.equal(a, b) for j, outs in got for a, b in zip(want[i][j], outs) if a is not None)

    for _ in range(3):
        with ThreadPoolExecutor(len(work)) as pool:
            assert all(pool.map(run, range(len(work))))
    assert wan.device_status() == wan.WAN_OK

// Linear layer with bias, activation and residual (wan_linear):
//
//     out[m, n] = act((sum_k a[m, k] w[n, k]) [a_scale[m] w_scale[n]] + bias[n]) + residual[m, n]
//
// on bf16 operands or e4m3 codes. This file holds the kernel for few rows: the
// WEIGHT rows are the 128-row operand of tcgen05.mma and the tokens its
// columns (N = 16 .. 128), so a call with one token pads it to 16 columns and
// not to a 128-row tile. What bounds it is the stream of weights from HBM:
// each CTA keeps a ring of TMA stages (128 weight rows x 128 bytes of K, and
// the same K of its tokens) in flight, and K is split over the CTAs of a
// cluster until every SM has a share of the stream. A thread of the epilogue
// holds one weight row (TMEM lane) and its tokens (columns). Without a split it
// finishes them from registers; with one, groups of 4 tokens are dealt out over
// the cluster and every CTA sends its float32 sums of a group straight from
// registers into the owner's shared memory (st.async, counted on the owner's
// mbarrier; the ring's memory, free once the cluster's products are done), where
// the same thread adds them in rank order: no workspace, no atomics, and a
// result that does not depend on timing.
//
// A call is launched so that it may start while the kernel before it on the
// stream still runs, and lets a call after it start early in turn: launch,
// barrier set-up and TMEM allocation then overlap the last CTAs of the kernel
// before (one after another 1 x 5120 x 5120 takes 13.2 us, 16.4 without). Every
// thread passes early_wait() before its first access to global memory, which
// holds until the kernels before are done and their writes visible. (On the norm
// and on CTA pairs, whose CTAs fill an SM, it cost time: 93600 x 128 10.7 ->
// 13.2 us, 512 x 5120 x 4096 32.8 -> 33.2.)
//
// Measured (in a captured graph and call after call alike): 1 x 5120 x 5120 bf16
// 12.7 us (4.1 TB/s of weights; 8.0 at the copy's rate, and a launch is 2.5), 24 x
// 13824 x 5120 e4m3 16.4 us (4.3 TB/s), 333 x 1003 x 1000 8.7 us. Library products
// of these sizes take 11.7, 14.1 and 4.7. Whole CTAs fall on the SMs: the 240 CTAs of
// the first leave the longest SM 23% more steps than the mean, the 216 of the second
// 37%. The third is a launch, one trip to memory, the sums' exchange and the epilogue.
#include "common.cuh"
#include "linear.cuh"
#include "sm100.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

namespace wan {

namespace {
using namespace sm100;

constexpr int WROWS = 128;                   // weight rows of a tile
constexpr int ROW_BYTES = 128;               // bytes of K per stage row (64 bf16 or 128 e4m3)
constexpr int W_BYTES = WROWS * ROW_BYTES;   // 16 KB
constexpr int MAX_STAGES = 12;
constexpr int THREADS = 192;                 // producer, MMA, 4 epilogue warps (one per quarter of the TMEM lanes)
constexpr int GROUP = 4;                     // tokens that travel and are finished together
constexpr int GROUP_BYTES = WROWS * GROUP * 4;
constexpr int SMEM_MAX = 225 * 1024;

__device__ __forceinline__ void early_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void early_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct SplitParams {
  int M, N, num_k, split;
  int mt, stages, chunk, tmem_cols;          // tokens per tile, ring, K steps per accumulator
  int recv;                                  // offset of the receive area; 0: the ring's memory
  uint32_t idesc;
  LinEpilogue e;
  int *watchdog;
};

// 16 tokens of one weight row n that a thread finishes together: group i + k of
// 4 tokens is group rank + split (i + k) of the tile. The loads do not look at
// what they are for until all of them are under way (tokens and columns past
// the end read the last ones).
template <bool F8>
struct Finish {
  const LinEpilogue &e;
  int m0, rows, n, N, rank, split;
  float bias, ws;
  float res[16], as[16];

  __device__ __forceinline__ int token(int i, int j) const { return (rank + split * (i + j / GROUP)) * GROUP + j % GROUP; }

  __device__ __forceinline__ void fetch(int i) {
    if (token(i, 0) >= rows) return;
    if (F8) {
#pragma unroll
      for (int j = 0; j < 16; ++j) as[j] = e.a_scale[m0 + min(token(i, j), rows - 1)];
    }
    if (!e.res) {
#pragma unroll
      for (int j = 0; j < 16; ++j) res[j] = 0.f;
      return;
    }
    const long long at = (long long)m0 * e.ldr + min(n, N - 1);
    if (e.res_f32) {
      const float *p = static_cast<const float *>(e.res) + at;
#pragma unroll
      for (int j = 0; j < 16; ++j) res[j] = p[min(token(i, j), rows - 1) * e.ldr];
    } else {
      const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(e.res) + at;
      __nv_bfloat16 h[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) h[j] = p[min(token(i, j), rows - 1) * e.ldr];
#pragma unroll
      for (int j = 0; j < 16; ++j) res[j] = __bfloat162float(h[j]);
    }
  }

  __device__ __forceinline__ void store(int i, float (&v)[16]) const {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = F8 ? fmaf(v[j], as[j] * ws, bias) : v[j] + bias;
    lin_act_row(v, e.act);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] += res[j];
    if (n >= N) return;
    const long long at = (long long)m0 * e.ldo + n;
    if (e.out_f32) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float *p = static_cast<float *>(e.out) + at + token(i, j) * e.ldo;
        if (token(i, j) < rows && WAN_DBG_OK(p, 4, e.out, e.out_hi, e.dbg, WAN_DBG_CODE_BASE + 17)) *p = v[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(e.out) + at + token(i, j) * e.ldo;
        if (token(i, j) < rows && WAN_DBG_OK(p, 2, e.out, e.out_hi, e.dbg, WAN_DBG_CODE_BASE + 17))
          *p = __float2bfloat16_rn(v[j]);
      }
    }
  }
};

// T tokens of this lane's weight row from TMEM column `col` on, the accumulators added
template <int T>
__device__ __forceinline__ void accumulators(uint32_t tmem, int col, int naccs, int mt, float (&v)[T]) {
  static_assert(T == 16, "one tcgen05.ld");
  uint32_t r[T];
  tmem_ld16(tmem + col, r);
  tmem_ld_wait();
#pragma unroll
  for (int j = 0; j < T; ++j) v[j] = __uint_as_float(r[j]);
  for (int a = 1; a < naccs; ++a) {
    tmem_ld16(tmem + a * mt + col, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < T; ++j) v[j] += __uint_as_float(r[j]);
  }
}

template <bool F8>
__global__ void __launch_bounds__(THREADS)
linear_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                    const SplitParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES], done, arrived;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = W_BYTES + p.mt * ROW_BYTES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = p.split, rank = blockIdx.x % split;   // cluster rank: the cluster spans x
  const int n0 = (blockIdx.x / split) * WROWS;
  const int m0 = blockIdx.y * p.mt;
  const int kb0 = (int)((long long)p.num_k * rank / split);
  const int nkb = (int)((long long)p.num_k * (rank + 1) / split) - kb0;
  const int rows = min(p.mt, p.M - m0);
  const int groups = (rows + GROUP - 1) / GROUP;
  const int mine = groups > rank ? (groups - rank - 1) / split + 1 : 0;   // groups rank, rank + split, ...

  auto load = [&](int i, int stage) {          // one step of K into a stage
    const uint32_t fb = smem_u32(&full[stage]), dst = smem_u32(smem + stage * stage_bytes);
    mbar_arrive_expect_tx(fb, stage_bytes);
    const int kx = (kb0 + i) * (F8 ? 128 : 64);
    tma_load_2d(dst, &tmW, kx, n0, fb);
    tma_load_2d(dst + W_BYTES, &tmA, kx, m0, fb);
  };
  const int ahead = min(p.stages, nkb);                 // loads that need no free stage
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(&done), 1);
    mbar_init(smem_u32(&arrived), 1);
    abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
    early_wait();
    for (int i = 0; i < ahead; ++i) load(i, i);
    // the other CTAs' sums of this CTA's groups
    mbar_arrive_expect_tx(smem_u32(&arrived), (split - 1) * mine * GROUP_BYTES);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), p.tmem_cols);
    tmem_relinquish();
  }
  early_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  early_next();               // not before the TMEM is there: the next kernel's CTAs may take what is left
  // Before sums travel, a barrier of the cluster says that every CTA's barriers
  // and receive area can be written: at once, or when the ring is free.
  const bool early = p.recv != 0;
  if (split > 1 && early) cluster_arrive();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    int stage = ahead == p.stages ? 0 : ahead, issued = ahead;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = ahead; i < nkb; ++i) {
      mbar_wait_lanes(ok, smem_u32(&empty[stage]), phase, &abort_flag, p.watchdog, 0x201);
      if (elect_one() && ok) load(i, stage);
      if (ok) ++issued;
      if (++stage == p.stages) { stage = 0; phase ^= 1; }
    }
    // every copy issued has landed before the CTA ends
    if (elect_one()) {
      int never = 0;
      for (int s = 0; s < p.stages; ++s) {
        const int fills = issued > s ? (issued - 1 - s) / p.stages + 1 : 0;
        if (fills > 0) mbar_wait(smem_u32(&full[s]), (fills - 1) & 1, &never, p.watchdog, 0x202);
      }
    }
    __syncwarp();
    if (split > 1) {
      if (!early) cluster_arrive();
      cluster_wait();
      cluster_arrive();
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t ring = smem_u32(smem), f0 = smem_u32(full);
    bool next = mbar_try_wait(f0, 0);
    for (int i = 0, in_chunk = 0, acc = 0; i < nkb; ++i) {
      if (!next) mbar_wait_lanes(ok, f0 + 8 * stage, phase, &abort_flag, p.watchdog, 0x211);
      tc_fence_after();
      const uint32_t base = ring + stage * stage_bytes;
      const uint64_t aw = desc_kmajor_sw128(base);
      const uint64_t bt = desc_kmajor_sw128(base + W_BYTES);
      const uint32_t d = tmem + acc * p.mt, eb = smem_u32(empty) + 8 * stage;
      if (++stage == p.stages) { stage = 0; phase ^= 1; }
      next = i + 1 < nkb && mbar_try_wait(f0 + 8 * stage, phase);     // asked ahead of the products' issue
      if (elect_one() && ok) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {       // 32 bytes of K each: + 2 in 16-byte units
          const uint32_t add = (in_chunk | kk) != 0;
          if (F8) mma_ss_f8(d, aw + 2 * kk, bt + 2 * kk, p.idesc, add);
          else mma_ss(d, aw + 2 * kk, bt + 2 * kk, p.idesc, add);
        }
        tc_commit(eb);
      }
      if (++in_chunk == p.chunk) { in_chunk = 0; ++acc; }
    }
    if (elect_one() && ok) tc_commit(smem_u32(&done));
    __syncwarp();
    if (split > 1) {
      if (!early) cluster_arrive();
      cluster_wait();
      cluster_arrive();
    }
  } else {
    // ------------------------------------------------ epilogue: weight row n, tokens m0 ..
    const LinEpilogue &e = p.e;
    const int q = warp & 3;                  // TMEM lanes this warp may read
    const int wrow = q * 32 + lane, n = n0 + wrow;
    const int naccs = (nkb + p.chunk - 1) / p.chunk;
    const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16);
    if (threadIdx.x == 64 && p.watchdog && *reinterpret_cast<volatile int *>(p.watchdog)) abort_flag = 1;   // an earlier launch gave up
    const float bias = e.bias && n < p.N ? __bfloat162float(e.bias[n]) : 0.f;
    const float ws = F8 && n < p.N ? e.w_scale[e.w_scale_rows ? n : 0] : 1.f;
    Finish<F8> f{e, m0, rows, n, p.N, rank, split, bias, ws};
    f.fetch(0);
    bool ok = mbar_wait_warp(smem_u32(&done), 0, &abort_flag, p.watchdog, 0x221);
    tc_fence_after();
    // sums from rank r of the i-th group of this CTA: recv + (r * most + i) * GROUP_BYTES
    const int most = (groups + split - 1) / split;
    uint8_t *recv = smem + p.recv + wrow * 16;
    if (split > 1) {
      if (!early) cluster_arrive();
      cluster_wait();
      // A CTA that gave up sends zeros, and waits for the others' sums like the
      // rest: nothing is on its way to a CTA that has ended.
      for (int c = 0; c < rows; c += 16) {
        float v[16] = {};
        if (ok) accumulators(taddr, c, naccs, p.mt, v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int g = c / GROUP + k, owner = g % split;
          if (g >= groups) break;
          const float4 s4 = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          uint8_t *at = recv + (rank * most + g / split) * GROUP_BYTES;
          if (owner == rank) *reinterpret_cast<float4 *>(at) = s4;
          else st_async_cluster(mapa_shared(smem_u32(at), owner), s4, mapa_shared(smem_u32(&arrived), owner));
        }
      }
      cluster_arrive();                      // nothing more leaves this warp
      if (mine > 0) {
        int never = 0;
        if (!mbar_wait_cluster(smem_u32(&arrived), 0, &never, p.watchdog, 0x222)) ok = false;
      }
    }
    if (ok) {
      for (int i = 0; i < mine; i += 4) {
        float v[16];
        if (split == 1) {
          accumulators(taddr, i * GROUP, naccs, p.mt, v);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = 0.f;
          for (int r = 0; r < split; ++r) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 x = *reinterpret_cast<const float4 *>(recv + (r * most + min(i + k, mine - 1)) * GROUP_BYTES);
              v[4 * k] += x.x; v[4 * k + 1] += x.y; v[4 * k + 2] += x.z; v[4 * k + 3] += x.w;
            }
          }
        }
        f.store(i, v);
        f.fetch(i + 4);
      }
    }
    tc_fence_before();
  }
  if (split > 1) cluster_wait();              // no CTA ends while another still sends to it
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
}

// ---------------------------------------------------------------- plan
// How a call is cut up: tokens per tile, K split.
struct Cut {
  int mt, split;
};
struct Plan {
  Cut c;
  int stages, smem, chunk, tmem_cols, recv;
};

constexpr int CTA_EXTRA = 1024 + 256;                          // shared memory that a CTA takes besides its ring
constexpr int SMS = 148;

int round_up(int v, int m) { return (v + m - 1) / m * m; }
int stage_of(const Cut &c) { return W_BYTES + c.mt * ROW_BYTES; }
int recv_bytes(const Cut &c) { return c.split > 1 ? (c.mt / GROUP + c.split - 1) / c.split * c.split * GROUP_BYTES : 0; }
long long ctas_of(const LinArgs &g, const Cut &c) {
  return (long long)((g.N + WROWS - 1) / WROWS) * c.split * ((g.M + c.mt - 1) / c.mt);
}
// Clusters of `split` CTAs that the card holds at once with one CTA to an SM: a
// GPC's SMs are not filled to the last one (16 clusters of 8 took two waves, 22
// of 6 one), so the runtime is asked, once for a device. It does not count
// several CTAs of a kernel to an SM; r of them make room for r times as many
// (40 clusters of 6 fit in two to an SM, 40 of 7 did not).
constexpr int MAX_SPLIT = 8, MAX_RESIDENT = 3;
struct Capacity {
  int clusters[MAX_SPLIT + 1];
};
const Capacity &capacity();
// CTAs of the grid that share an SM
int ctas_per_sm(const LinArgs &g, const Cut &c) {
  const long long clusters = ctas_of(g, c) / c.split;
  const int room = capacity().clusters[c.split];
  return (int)((clusters + room - 1) / room);
}
// Accumulators of a CTA: one for every part of its K (lin_parts), as many as go
// into its share of TMEM while a part then stays below 16 steps, else into all of it
int accumulators_of(const LinArgs &g, int num_k, const Cut &c) {
  const int nkb = (num_k + c.split - 1) / c.split, want = lin_parts(g, nkb), share = TMEM_SHARE / c.mt;
  return std::min(want, nkb <= 16 * share ? share : 512 / c.mt);
}
// TMEM columns of a CTA, and the shared memory that goes with its share of them
// (sm100.cuh, SMEM_ALONE)
constexpr int SMEM_SHARE = SM_SMEM / 4 - CTA_EXTRA;
int columns_of(const LinArgs &g, int num_k, const Cut &c) {
  int cols = TMEM_SHARE;
  while (cols < accumulators_of(g, num_k, c) * c.mt) cols *= 2;
  return cols;
}
// CTAs that an SM holds at once: all of its own while each keeps three stages
int resident(const LinArgs &g, int num_k, const Cut &c) {
  if (columns_of(g, num_k, c) > TMEM_SHARE) return 1;
  const int fit = SM_SMEM / (3 * stage_of(c) + 1024 + CTA_EXTRA);
  return std::min(std::min(fit, MAX_RESIDENT), ctas_per_sm(g, c));
}

Plan make_plan(const LinArgs &g, int num_k, const Cut &c) {
  const int nkb = (num_k + c.split - 1) / c.split;
  const int nacc = accumulators_of(g, num_k, c), cols = columns_of(g, num_k, c);
  const int stage = stage_of(c);
  // few tokens: a receive area of its own (8 to 28 KB) saves a barrier after the
  // products (14.6 -> 13.4 us at 1 x 5120 x 5120), unless it would leave the ring
  // fewer than three stages, as it does for 17 to 32 tokens with three CTAs on an
  // SM: 26 x 13304 x 11216 65.4 us with it and two stages, 59.2 without and with
  // three, 20 x 12000 x 4096 22.0 and 21.2
  const int room = std::min(SM_SMEM / resident(g, num_k, c) - CTA_EXTRA, SMEM_MAX) - 1024;
  int own = c.split > 1 && c.mt <= 32 ? recv_bytes(c) : 0;
  if ((room - own) / stage < std::min(3, nkb)) own = 0;
  int stages = (room - own) / stage;
  stages = std::max(2, std::min(std::min(stages, nkb), MAX_STAGES));
  int smem = (own ? stages * stage + own : std::max(stages * stage, recv_bytes(c))) + 1024;
  smem = std::max(smem, cols > TMEM_SHARE ? SMEM_ALONE : SMEM_SHARE);
  return Plan{c, stages, smem, (nkb + nacc - 1) / nacc, cols, own ? stages * stage : 0};
}

// Time of a cut in SM cycles, to compare cuts and kernels by: a start and an
// end, the sums' way through the cluster, what an SM takes in for its CTAs, and
// a new start and epilogue for every further wave. Measured: an SM takes in 28
// bytes a cycle from HBM (22 with one CTA) and 55 from L2 (an operand comes from
// HBM for the first tile that reads it), and the card 3400 from HBM; SM and CTAs
// need 400 cycles for a step of K at least; a token costs the epilogue 45, 70
// with a residual. The cut or pair tile taken by these two costs was 1 to 3%
// slower in the mean than the best of all, over six sets of 26 random sizes; the
// worst of the last 52 by 37% (735 x 2052 x 592: pair tiles 11.7 us, tiles of 48
// tokens 8.5), four more by 5 to 15%.
double split_cost(const LinArgs &g, int num_k, const Cut &c) {
  const double ntn = (g.N + WROWS - 1) / WROWS, ntm = (g.M + c.mt - 1) / c.mt;
  const double per_sm = ctas_per_sm(g, c);
  const int nkb = (num_k + c.split - 1) / c.split;
  const double hbm = per_sm > 1.0 ? 28.0 : 22.0;
  auto ingest = [&](double bytes, double readers) { return bytes * (1.0 / hbm / readers + (1.0 - 1.0 / readers) / 55.0); };
  const double step = ingest(W_BYTES, ntm) + ingest((double)std::min(c.mt, g.M) * ROW_BYTES, ntn);
  const double dram = ((double)g.M + g.N) * g.K * (g.fp8 ? 1 : 2) / 3400.0;
  const double waves = ceil(per_sm / resident(g, num_k, c)), finish = (g.res ? 70.0 : 45.0) * c.mt / (c.split > 1 ? 2.0 : 1.0);
  return 8500.0 + waves * finish + (800.0 + 10.0 * c.mt) * (per_sm - 1.0) + (c.split > 1 ? 4000.0 + 100.0 * c.split : 0.0) +
         4000.0 * (waves - 1.0) + std::max(std::max(per_sm * step, 400.0) * nkb, dram);
}
// The same of the pair kernel: tiles of 256 x bn in rounds of 74 pairs. A step
// of K takes its products (2 bn cycles) or its operands' way onto the SM (60
// bytes a cycle, 28 from HBM: measured 560 cycles at bn = 256, 444 at 160), a
// tile no less than its epilogue (9000 cycles at bn = 256, more with a residual,
// 23000 and 31000 where the rows of out or residual are out of the TMA unit's
// reach); the last one is in the open.
double pair_cost(const LinArgs &g, int num_k, int bn) {
  const double tiles = ceil(g.M / 256.0) * ceil(g.N / (double)bn);
  const LinEpilogue e = lin_epilogue(g);
  const double epi = 3000.0 + (e.vec_out && e.vec_res ? (g.res ? 8500.0 : 6000.0) : (g.res ? 28000.0 : 20000.0)) * bn / 256.0;
  // bytes of a step that no other tile has brought into L2
  const double cold = 64.0 * bn / ceil(g.M / 256.0) + W_BYTES * std::min(1.0, g.M / 256.0) / ceil(g.N / (double)bn);
  const double step = std::max(2.0 * bn, cold / 28.0 + std::max(0.0, W_BYTES + 64.0 * bn - cold) / 60.0);
  const double rounds = ceil(tiles / 74.0);
  return 10000.0 + num_k * step + epi + (rounds - 1.0) * std::max(num_k * step, epi);
}

// The kernel of a call: pair_bn != 0 for the pair kernel, else the plan.
struct Choice {
  int pair_bn;
  Plan plan;
};
Choice choose(const LinArgs &g) {
  const int num_k = (g.K + (g.fp8 ? 128 : 64) - 1) / (g.fp8 ? 128 : 64);
  Cut cut = {};
  double best = 0.0;
  for (int want = 16; want <= 128; want += 16) {
    if (want > 16 && want - 16 >= g.M) break;
    const int tiles = (g.M + want - 1) / want, mt = round_up((g.M + tiles - 1) / tiles, 16);
    if (tiles > 65535) continue;
    for (int split = 1; split <= std::min(MAX_SPLIT, num_k); ++split) {
      const Cut c = {mt, split};
      // parts of K no longer than the longest on CTA pairs
      const int nkb = (num_k + split - 1) / split;
      if (lin_parts(g, nkb) > 1 && nkb > 32 * accumulators_of(g, num_k, c)) continue;
      const double cost = split_cost(g, num_k, c);
      if (!cut.mt || cost < best) { best = cost; cut = c; }
    }
  }
  int bn = 0;
  for (int n = lin_pair_parts(g, num_k) > 1 ? LIN_PARTS_BN : 256; n >= 96; n -= 32) {
    const double cost = pair_cost(g, num_k, n);
    if ((!cut.mt && !bn) || cost < best) { best = cost; bn = n; }
  }
  return bn ? Choice{bn, Plan{}} : Choice{0, make_plan(g, num_k, cut)};
}

template <bool F8>
int set_attributes() {
  static std::atomic<uint64_t> ready{0};       // devices whose attributes are set
  int dev = 0;
  WAN_TRY_CUDA(cudaGetDevice(&dev), "linear device");
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    WAN_TRY_CUDA(cudaFuncSetAttribute(linear_split_kernel<F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX),
                 "linear smem attribute");
    WAN_TRY_CUDA(cudaFuncSetAttribute(linear_split_kernel<F8>, cudaFuncAttributePreferredSharedMemoryCarveout, 100),
                 "linear smem carveout");
    if (dev < 64) ready.fetch_or(uint64_t(1) << dev);
  }
  return WAN_OK;
}

// Where the runtime gives no answer, 7/8 of the SMs count.
const Capacity &capacity() {
  static Capacity known[64];
  static std::once_flag once[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  std::call_once(once[dev], [&] {
    const bool ask = set_attributes<false>() == WAN_OK;
    for (int split = 1; split <= MAX_SPLIT; ++split) {
      int n = SMS / split;
      if (split > 1) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = split; attr[0].val.clusterDim.y = 1; attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)(split * SMS), 1, 1);
        cfg.blockDim = dim3(THREADS, 1, 1);
        cfg.dynamicSmemBytes = SMEM_MAX;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int got = 0;
        if (ask && cudaOccupancyMaxActiveClusters(&got, linear_split_kernel<false>, &cfg) == cudaSuccess && got > 0) n = got;
        else n = n * 7 / 8;
      }
      known[dev].clusters[split] = n;
    }
    cudaGetLastError();                        // a refused question is no error of the call
  });
  return known[dev];
}

template <bool F8>
int launch(const LinArgs &g, const Plan &pl, cudaStream_t s) {
  if (const int bad = set_attributes<F8>()) return bad;
  CUtensorMap tw, ta;
  int rc;
  if (F8) {
    if ((rc = encode_tmap_2d_u8(&tw, g.w, g.K, g.N, (uint64_t)g.ldw, 128, WROWS))) return rc;
    if ((rc = encode_tmap_2d_u8(&ta, g.a, g.K, g.M, (uint64_t)g.lda, 128, pl.c.mt))) return rc;
  } else {
    if ((rc = encode_tmap_2d_bf16(&tw, g.w, g.K, g.N, (uint64_t)g.ldw * 2, 64, WROWS))) return rc;
    if ((rc = encode_tmap_2d_bf16(&ta, g.a, g.K, g.M, (uint64_t)g.lda * 2, 64, pl.c.mt))) return rc;
  }
  SplitParams p = {};
  p.M = g.M; p.N = g.N; p.num_k = (g.K + (F8 ? 128 : 64) - 1) / (F8 ? 128 : 64); p.split = pl.c.split;
  p.mt = pl.c.mt; p.stages = pl.stages; p.chunk = pl.chunk; p.recv = pl.recv; p.tmem_cols = pl.tmem_cols;
  p.idesc = F8 ? idesc_e4m3(WROWS, pl.c.mt) : idesc_bf16(WROWS, pl.c.mt, 0);
  p.e = lin_epilogue(g);
  p.watchdog = watchdog_ptr();
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = pl.c.split; attr[0].val.clusterDim.y = 1; attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  const int tiles = (g.M + pl.c.mt - 1) / pl.c.mt;
  cfg.gridDim = dim3((unsigned)(ctas_of(g, pl.c) / tiles), (unsigned)tiles, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  WAN_TRY_CUDA(cudaLaunchKernelEx(&cfg, linear_split_kernel<F8>, tw, ta, p), "linear launch");
  return WAN_OK;
}

int launch_plan(const LinArgs &g, const Plan &pl, cudaStream_t s) {
  return g.fp8 ? launch<true>(g, pl, s) : launch<false>(g, pl, s);
}
}  // namespace

int launch_linear(const LinArgs &g, cudaStream_t s) {
  // the choice costs a few microseconds of the host: it is kept in one of 32 slots,
  // by all that it is made from (sizes, types, the rows' alignment, a residual, the
  // card); sizes of one slot displace each other
  struct Known {
    const Capacity *card;
    int M, N, K, kind;
    Choice choice;
  };
  thread_local Known known[32] = {};
  const LinEpilogue e = lin_epilogue(g);
  const int kind = 1 | (g.fp8 ? 2 : 0) | (g.out_f32 ? 4 : 0) | (e.vec_out && e.vec_res ? 8 : 0) | (g.res ? 16 : 0);
  const unsigned h = ((unsigned)g.M * 2654435761u ^ (unsigned)g.N * 40503u ^ (unsigned)g.K * 65599u ^ (unsigned)kind) >> 3;
  Known &k = known[h % 32];
  const Capacity *card = &capacity();
  if (k.card != card || k.M != g.M || k.N != g.N || k.K != g.K || k.kind != kind) {
    k = Known{card, g.M, g.N, g.K, kind, choose(g)};
  }
  return k.choice.pair_bn ? gemm_tc_linear(g, k.choice.pair_bn, s) : launch_plan(g, k.choice.plan, s);
}

}  // namespace wan

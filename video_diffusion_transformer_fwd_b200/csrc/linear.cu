// Linear layer with bias, activation and residual (wan_linear):
//
//     out[m, n] = act((sum_k a[m, k] w[n, k]) [a_scale[m] w_scale[n]] + bias[n]) + residual[m, n]
//
// on bf16 operands or e4m3 codes. This file holds the kernel for few rows: the
// WEIGHT rows are the 128-row operand of tcgen05.mma and the tokens its
// columns (N = 16 .. 256), so a call with one token pads it to 16 columns and
// not to a 128-row tile. What bounds it is the stream of weights from HBM:
// each CTA keeps a ring of TMA stages (128 weight rows x 128 bytes of K, and
// the same K of its tokens) in flight, and K is split over the CTAs of a
// cluster until every SM has a share of the stream. The CTAs' partial sums
// (float32, in shared memory as [token][128]) are added through distributed
// shared memory in rank order, so the result does not depend on timing and no
// workspace is needed; scales, bias, activation and residual are applied
// there, on rows of 128 consecutive outputs.
#include "common.cuh"
#include "linear.cuh"
#include "sm100.cuh"

#include <atomic>
#include <cmath>

namespace wan {

namespace {
using namespace sm100;

constexpr int WROWS = 128;                   // weight rows of a tile
constexpr int ROW_BYTES = 128;               // bytes of K per stage row (64 bf16 or 128 e4m3)
constexpr int W_BYTES = WROWS * ROW_BYTES;   // 16 KB
constexpr int MAX_STAGES = 12;
constexpr int THREADS = 192;                 // producer, MMA, 4 epilogue warps
constexpr int SMEM_MAX = 225 * 1024;
constexpr int SMEM_HALF = 112 * 1024;        // two CTAs per SM

struct SplitParams {
  int M, N, num_k, split;
  int mt, stages, nacc, chunk, tmem_cols;    // tokens per tile, ring, accumulators, K steps per accumulator
  uint32_t idesc;
  LinEpilogue e;
  int *watchdog;
};

template <bool F8>
__global__ void __launch_bounds__(THREADS)
linear_split_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                    const SplitParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES], done;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int stage_bytes = W_BYTES + p.mt * ROW_BYTES;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % p.split;               // cluster rank: the cluster spans x
  const int n0 = (blockIdx.x / p.split) * WROWS;
  const int m0 = blockIdx.y * p.mt;
  const int kb0 = (int)((long long)p.num_k * rank / p.split);
  const int nkb = (int)((long long)p.num_k * (rank + 1) / p.split) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(&done), 1);
    // a wait of an earlier launch gave up: no work, but every barrier below is still passed
    abort_flag = (p.watchdog && *reinterpret_cast<volatile int *>(p.watchdog)) ? 1 : 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmA);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const bool skip = abort_flag != 0;

  if (warp == 0 && lane == 0 && !skip) {
    // ------------------------------------------------ TMA producer
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    for (; issued < nkb; ++issued) {
      if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1, &abort_flag, p.watchdog, 0x201)) break;
      const uint32_t fb = smem_u32(&full[stage]);
      mbar_arrive_expect_tx(fb, stage_bytes);
      const uint32_t dst = smem_u32(smem + stage * stage_bytes);
      const int kx = (kb0 + issued) * (F8 ? 128 : 64);
      tma_load_2d(dst, &tmW, kx, n0, fb);
      tma_load_2d(dst + W_BYTES, &tmA, kx, m0, fb);
      if (++stage == p.stages) { stage = 0; phase ^= 1; }
    }
    // every copy issued has landed before the stages are reused or the CTA ends
    int never = 0;
    for (int s = 0; s < p.stages; ++s) {
      const int fills = issued > s ? (issued - 1 - s) / p.stages + 1 : 0;
      if (fills > 0) mbar_wait(smem_u32(&full[s]), (fills - 1) & 1, &never, p.watchdog, 0x202);
    }
  } else if (warp == 1 && lane == 0 && !skip) {
    // ------------------------------------------------ MMA issuer
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = 0, in_chunk = 0, acc = 0; i < nkb; ++i) {
      if (!mbar_wait(smem_u32(&full[stage]), phase, &abort_flag, p.watchdog, 0x211)) { ok = false; break; }
      tc_fence_after();
      const uint32_t base = smem_u32(smem + stage * stage_bytes);
      const uint64_t aw = desc_kmajor_sw128(base);
      const uint64_t bt = desc_kmajor_sw128(base + W_BYTES);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {       // 32 bytes of K each: + 2 in 16-byte units
        const uint32_t d = tmem + acc * p.mt;
        if (F8) mma_ss_f8(d, aw + 2 * kk, bt + 2 * kk, p.idesc, (in_chunk | kk) != 0);
        else mma_ss(d, aw + 2 * kk, bt + 2 * kk, p.idesc, (in_chunk | kk) != 0);
      }
      tc_commit(smem_u32(&empty[stage]));
      if (++stage == p.stages) { stage = 0; phase ^= 1; }
      if (++in_chunk == p.chunk) { in_chunk = 0; ++acc; }
    }
    if (ok) tc_commit(smem_u32(&done));
  } else if (warp >= 2 && !skip) {
    // ------------------------------------------------ accumulators -> shared memory
    const bool ok = mbar_wait(smem_u32(&done), 0, &abort_flag, p.watchdog, 0x221);
    tc_fence_after();
    if (__all_sync(0xffffffffu, ok)) {
      // all products are done and their operands read: the ring's memory is free
      const int q = warp & 3;                // TMEM lanes this warp may read
      float *part = reinterpret_cast<float *>(smem) + q * 32 + lane;
      const int naccs = (nkb + p.chunk - 1) / p.chunk;
      const int cols = min(p.mt, p.M - m0);
      for (int c = 0; c < cols; c += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c, r);
        tmem_ld_wait();
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
        for (int a = 1; a < naccs; ++a) {
          tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + a * p.mt + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(r[j]);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * WROWS] = v[j];
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if (p.split > 1) cluster_sync_all(); else __syncthreads();
  tc_fence_after();

  // ------------------------------------------------ sum over the cluster, epilogue, stores
  if (!abort_flag) {
    const uint32_t part = smem_u32(smem);
    const int n = n0 + 4 * lane;
    const int rows = min(p.mt, p.M - m0);
    LinColumns col;
    if (n < p.N) col.load(p.e, n, p.N, F8);
    for (int t = rank + p.split * warp; t < rows; t += p.split * (THREADS / 32)) {
      const uint32_t off = part + (uint32_t)(t * WROWS + 4 * lane) * 4;
      float4 v;
      if (p.split > 1) {
        v = ld_shared_cluster_f4(mapa_shared(off, 0));
        for (int r = 1; r < p.split; ++r) {
          const float4 w = ld_shared_cluster_f4(mapa_shared(off, r));
          v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
        }
      } else {
        v = *reinterpret_cast<const float4 *>(smem + (off - part));
      }
      if (n < p.N) lin_store4(p.e, col, m0 + t, n, p.N, v, F8);
    }
  }
  if (p.split > 1) cluster_sync_all();        // the peers have read this CTA's sums
  if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
}

// ---------------------------------------------------------------- plan
struct Plan {
  int mt, split, stages, smem, nacc, chunk, tmem_cols;
};

int round_up(int v, int m) { return (v + m - 1) / m * m; }

Plan plan_of(const LinArgs &g) {
  const int num_k = (g.K + (g.fp8 ? 128 : 64) - 1) / (g.fp8 ? 128 : 64);
  const int nt = (g.N + WROWS - 1) / WROWS;
  Plan best = {};
  double best_cost = 0.0;
  // bf16 products are accumulated by the tensor core with a rounding toward
  // zero that grows with the number of steps (relative 1.1e-9 K, measured
  // against 64 bits): harmless under a bf16 output, but a float32 output gets
  // a new accumulator every 64 steps (4096 of K), added in float32
  const bool chained = !g.fp8 && g.out_f32;
  const int t0 = (g.M + 255) / 256;
  for (int t = t0; t <= t0 + 4; ++t) {
    const int mt = round_up((g.M + t - 1) / t, 16);
    if (t > t0 && mt < 16) break;
    const int tiles = (g.M + mt - 1) / mt;
    for (int split = 1; split <= 8; split *= 2) {
      if (split > num_k) break;
      const int nkb = (num_k + split - 1) / split;
      const int stage = W_BYTES + mt * ROW_BYTES;
      const int occ = 4 * stage + 1024 <= SMEM_HALF && mt * 512 + 1024 <= SMEM_HALF ? 2 : 1;
      const int budget = (occ == 2 ? SMEM_HALF : SMEM_MAX) - 1024;
      int stages = budget / stage;
      if (stages > MAX_STAGES) stages = MAX_STAGES;
      int nacc = chained ? (nkb + 63) / 64 : 1;
      const int most = 512 / occ / mt;
      if (nacc > most) nacc = most;
      const int chunk = (nkb + nacc - 1) / nacc;
      const double kstep = fmax(2.0 * mt, fmax(128.0 + mt, (W_BYTES + mt * 128.0) / 56.0));
      const double ctas = (double)nt * tiles * split;
      const double per_sm = ceil(ctas / 148.0);
      double cost = 4000.0 + per_sm * (nkb * kstep + (per_sm > occ ? 2000.0 : 0.0)) + 6.0 * mt * per_sm + (split > 1 ? 1500.0 : 0.0);
      const double dram = ((double)g.N + g.M) * g.K * (g.fp8 ? 1 : 2) / 3400.0 + 4000.0 + (split > 1 ? 1500.0 : 0.0);
      if (dram > cost) cost = dram;
      if (chained) cost *= 1.0 + 0.5 * (chunk > 64) ;
      if (best.mt == 0 || cost < best_cost) {
        best_cost = cost;
        int cols = 32;
        while (cols < nacc * mt) cols *= 2;
        int smem = stages * stage;
        if (smem < mt * 512) smem = mt * 512;
        best = Plan{mt, split, stages, smem + 1024, nacc, chunk, cols};
      }
    }
  }
  return best;
}

template <bool F8>
int launch(const LinArgs &g, const Plan &pl, cudaStream_t s) {
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
  CUtensorMap tw, ta;
  int rc;
  if (F8) {
    if ((rc = encode_tmap_2d_u8(&tw, g.w, g.K, g.N, (uint64_t)g.ldw, 128, WROWS))) return rc;
    if ((rc = encode_tmap_2d_u8(&ta, g.a, g.K, g.M, (uint64_t)g.lda, 128, pl.mt))) return rc;
  } else {
    if ((rc = encode_tmap_2d_bf16(&tw, g.w, g.K, g.N, (uint64_t)g.ldw * 2, 64, WROWS))) return rc;
    if ((rc = encode_tmap_2d_bf16(&ta, g.a, g.K, g.M, (uint64_t)g.lda * 2, 64, pl.mt))) return rc;
  }
  SplitParams p = {};
  p.M = g.M; p.N = g.N; p.num_k = (g.K + (F8 ? 128 : 64) - 1) / (F8 ? 128 : 64); p.split = pl.split;
  p.mt = pl.mt; p.stages = pl.stages; p.nacc = pl.nacc; p.chunk = pl.chunk; p.tmem_cols = pl.tmem_cols;
  p.idesc = F8 ? idesc_e4m3(WROWS, pl.mt) : idesc_bf16(WROWS, pl.mt, 0);
  p.e = lin_epilogue(g);
  p.watchdog = watchdog_ptr();
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = pl.split; attr[0].val.clusterDim.y = 1; attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)((g.N + WROWS - 1) / WROWS * pl.split), (unsigned)((g.M + pl.mt - 1) / pl.mt), 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  WAN_TRY_CUDA(cudaLaunchKernelEx(&cfg, linear_split_kernel<F8>, tw, ta, p), "linear launch");
  return WAN_OK;
}
}  // namespace

int launch_linear(const LinArgs &g, cudaStream_t s) {
  const Plan pl = plan_of(g);
  if ((g.M + pl.mt - 1) / pl.mt > 65535) return set_error(WAN_EINVAL, "linear: M=%d too large", g.M);
  return g.fp8 ? launch<true>(g, pl, s) : launch<false>(g, pl, s);
}

}  // namespace wan

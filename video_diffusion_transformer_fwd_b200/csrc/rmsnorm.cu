// Row RMS norm with the residual's addition (wan_rmsnorm):
//
//     h = x + r                       (h = x without a residual)
//     y = (h g) rstd,  rstd = 1 / sqrt(sum h^2 / D + eps)
//
// stored as bf16 / float32, or as e4m3 codes with one scale per row. x, r, h
// and y cross HBM once: a row stays on the SM between its reads and its
// writes, so the kernel is bound by those bytes alone.
//
// The sum of squares and the row's maximum are reduced together: rounding is
// monotone, so max |(h g) rstd| = fl(max |h g| * rstd) exactly, and the scale
// of the e4m3 output needs no second pass after rstd is known. h is the
// float32 sum, rounded only where it is stored (the norm sees the unrounded
// sum: one rounding less than adding, storing and reading back).
//
// Two kernels, by how the rows lie:
//   rmsnorm_kernel         8 elements a thread at a time, in registers from the
//                          loads to the stores; short rows share a warp. Where
//                          the row strides agree modulo 8 (all dense matrices),
//                          row `row` begins s = row ld mod 8 elements after a
//                          boundary of 8 in every matrix, so the groups
//                          8 c - s .. 8 c - s + 7 are aligned in all of them;
//                          only a row's first and last group are taken apart;
//   rmsnorm_ragged_kernel  strides that do not agree: a row comes in and leaves
//                          in whole 16-byte pieces of memory through shared
//                          memory, where its elements are picked at their own
//                          offsets (12000 x 3163 bf16: 82 us, 42 where the
//                          strides agree).
// Measured in a captured graph, inputs out of L2 (call after call): 32760 x 5120
// bf16 onto a float32 stream and into codes 264 us, 7.0 TB/s (288), 7800 x 1536 of
// the same 22.4, 5.9 TB/s (22.9), 93600 x 128 bf16 10.6, 4.5 TB/s (12.0), 2011 x 1037
// 7.4, 2.8 TB/s (8.2), one row of 5120 2.5 us, which is a launch (8.1: the host's
// work). Short calls are
// bound by the launch and one trip to memory; dense rows of odd width by the
// instructions that pick their elements.
#include "common.cuh"
#include "e4m3.cuh"

#include <float.h>

#include <atomic>

namespace wan {

namespace {

struct RmsArgs {
  int rows, D;
  const void *x; long long ldx;
  const void *r; long long ldr;
  const float *g; float eps;
  void *h; long long ldh;
  void *y; long long ldy;
  float *scale;
  int inner;                        // rows with 7 more elements of x and r behind their end
  int *dbg;
};

// 8 elements as they lie in memory (streaming: a row is read once). load_part:
// elements lo .. lo + 7 of a row of D, one by one, the row's ends in place of
// what lies outside it.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = __ldcs(reinterpret_cast<const float4 *>(p));
    b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void load_part(const float *row, int lo, int D) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = row[min(max(lo + e, 0), D - 1)];
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <> struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { u = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void load_part(const __nv_bfloat16 *row, int lo, int D) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = __bfloat16_as_ushort(row[min(max(lo + e, 0), D - 1)]);
    u = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
};

// Streaming stores: 1-3% over plain ones on every width measured.
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t *>(&b);
  }
  __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8_codes(uint8_t *p, const float (&v)[8], float inv) {
  __stcs(reinterpret_cast<uint2 *>(p), make_uint2(quant4(make_float4(v[0], v[1], v[2], v[3]), inv),
                                                  quant4(make_float4(v[4], v[5], v[6], v[7]), inv)));
}

// The gain of elements lo .. lo + 7. Rows that begin off a boundary of 8 (SHIFT)
// take the three aligned float4 around them and move their elements into place
// by the row's offset (12000 x 3163 bf16: 43 us, 65 with 8 single loads
// after the row);
// the groups at the row's ends, whose three would leave the gain, take single
// elements.
template <bool SHIFT> struct Gain8 {
  float4 p, q, r;
  __device__ __forceinline__ static int offset(int lo, int D) {
    return SHIFT && lo >= 0 && lo - (lo & 3) + 12 <= D ? lo & 3 : 0;
  }
  __device__ __forceinline__ void load(const float *g, int lo, int D) {
    if (!SHIFT || (lo >= 0 && lo - (lo & 3) + 12 <= D)) {
      const float4 *at = reinterpret_cast<const float4 *>(g + (SHIFT ? lo - (lo & 3) : lo));
      p = __ldg(at);
      q = __ldg(at + 1);
      if (SHIFT) r = __ldg(at + 2);
    } else {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = __ldg(g + min(max(lo + e, 0), D - 1));
      p = make_float4(w[0], w[1], w[2], w[3]);
      q = make_float4(w[4], w[5], w[6], w[7]);
      r = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void apply(float (&v)[8], int lo, int D) const {
    float w[11] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w, 0.f, 0.f, 0.f};
    if constexpr (SHIFT) {
      w[8] = r.x; w[9] = r.y; w[10] = r.z;
      const int off = offset(lo, D);
#pragma unroll
      for (int e = 0; e < 10; ++e) w[e] = off & 1 ? w[e + 1] : w[e];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = off & 2 ? w[e + 2] : w[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= w[e];
  }
};

template <typename T>
__device__ __forceinline__ void store_part(T *row, int lo, int D, const float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (lo + e >= 0 && lo + e < D) ElemIO<T>::store(row + lo + e, v[e]);
}
__device__ __forceinline__ void store_part_codes(uint8_t *row, int lo, int D, const float (&v)[8], float inv) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (lo + e >= 0 && lo + e < D) row[lo + e] = __nv_cvt_float_to_fp8(__fmul_rn(v[e], inv), __NV_SATFINITE, __NV_E4M3);
}

// 1 / rms of the row, and for codes the row's scale (written by one thread)
// and the factor from y to a code.
struct RowFactors {
  float rstd, inv;
  template <bool CODES>
  static __device__ __forceinline__ RowFactors of(const RmsArgs &a, long long row, float ss, float top, bool writer) {
    RowFactors f;
    f.rstd = 1.0f / sqrtf(ss / (float)a.D + a.eps);
    f.inv = 1.f;
    if constexpr (CODES) {
      const float amax = top * f.rstd;
      f.inv = fminf(e4m3_inv_scale(amax), FLT_MAX);   // amax below 448 / FLT_MAX: no infinite factor
      if (!(amax == amax)) f.inv = amax;              // a row with NaN: every code NaN
      if (writer && WAN_DBG_OK(a.scale + row, 4, a.scale, a.scale + a.rows, a.dbg, WAN_DBG_CODE_BASE + 13))
        a.scale[row] = __fdiv_rn(amax, E4M3_MAX);
    }
    return f;
  }
};

// Sum and maximum over the CTA (one barrier).
template <bool CODES>
__device__ __forceinline__ void cta_reduce(float &ss, float &top, float (&red)[2][32]) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
  ss = warp_sum(ss);
  if constexpr (CODES) top = warp_max(top);
  if (lane == 0) {
    red[0][wid] = ss;
    if constexpr (CODES) red[1][wid] = top;
  }
  __syncthreads();
  ss = warp_sum(lane < nw ? red[0][lane] : 0.f);
  if constexpr (CODES) top = warp_max(lane < nw ? red[1][lane] : 0.f);
}

constexpr int ROW_CTA = 128;          // threads of a CTA that holds several rows
constexpr int VEC_CTA = RMS_MAX_D / 32;

// TPR threads of one warp per row (several rows per CTA), or TPR = 0: the
// whole CTA per row. NV groups of 8 elements per thread; with 4 of them
// registers are held to what lets two CTAs share an SM. SHIFT: rows do not all
// begin on a boundary of 8 elements.
template <typename XT, typename RT, bool RES, typename YT, int NV, int TPR, bool SHIFT>
__global__ void __launch_bounds__(TPR ? ROW_CTA : VEC_CTA, !TPR && NV == 4 ? 2 : 1) rmsnorm_kernel(const RmsArgs a) {
  constexpr bool CODES = sizeof(YT) == 1;
  __shared__ float red[2][32];
  const int tpr = TPR ? TPR : blockDim.x;
  const int t = TPR ? (int)(threadIdx.x % TPR) : (int)threadIdx.x;
  const long long row = TPR ? (long long)blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR : blockIdx.x;
  const bool live = row < a.rows;     // all lanes of a warp take part in the shuffles
  const int D = a.D;
  const int shift = SHIFT ? (int)((row * a.ldx) & 7) : 0;
  const int nv = (D + shift + 7) / 8;
  // group c: elements lo .. lo + 7
  auto lo_of = [&](int c) { return 8 * c - shift; };
  auto whole = [&](int c) { return !SHIFT || (lo_of(c) >= 0 && lo_of(c) + 8 <= D); };
  float v[NV][8];
  float ss = 0.f, top = 0.f;
  Raw8<XT> xv[NV];
  Raw8<RT> rv[NV];
  // The gain, which every row reads from the caches, comes with the row where
  // registers allow (32760 x 5120 onto codes: 263 us, 271 when it was read after
  // the row; rows of a warp are faster so: 93600 x 128 10.7 us, 12.1 with it).
  constexpr bool EARLY = TPR == 0 && NV <= 2;
  Gain8<SHIFT> gv[NV];
  if (live) {
    // all loads of the row before the first use of one
    const XT *xr = static_cast<const XT *>(a.x) + row * a.ldx;
    const RT *rr = RES ? static_cast<const RT *>(a.r) + row * a.ldr : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * tpr;
      if (c < nv) {
        // a group that reaches into the neighbouring rows is read with them,
        // except where it would reach behind the matrix
        if (!SHIFT || lo_of(c) + 8 <= D || row < a.inner) {
          xv[i].load(xr + lo_of(c));
          if constexpr (RES) rv[i].load(rr + lo_of(c));
        } else {
          xv[i].load_part(xr, lo_of(c), D);
          if constexpr (RES) rv[i].load_part(rr, lo_of(c), D);
        }
      }
    }
    if (EARLY && a.g) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (t + i * tpr < nv) gv[i].load(a.g, lo_of(t + i * tpr), D);
    }
    RT *hr = RES && a.h ? static_cast<RT *>(a.h) + row * a.ldh : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * tpr;
      if (c < nv) {
        const int lo = lo_of(c);
        xv[i].get(v[i]);
        if constexpr (RES) {
          float q[8];
          rv[i].get(q);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] += q[e];
        }
        if constexpr (SHIFT) {
          if (!whole(c)) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (lo + e < 0 || lo + e >= D) v[i][e] = 0.f;
          }
        }
        if constexpr (RES) {
          if (hr && WAN_DBG_OK(hr + max(lo, 0), (min(lo + 8, D) - max(lo, 0)) * sizeof(RT), a.h,
                               static_cast<RT *>(a.h) + (a.rows - 1) * a.ldh + D, a.dbg, WAN_DBG_CODE_BASE + 12)) {
            if (whole(c)) store8(hr + lo, v[i]);
            else store_part(hr, lo, D, v[i]);
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
        if (a.g) {
          if (!EARLY) gv[i].load(a.g, lo, D);
          gv[i].apply(v[i], lo, D);
        }
        if constexpr (CODES) {
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[i][e]));
        }
      }
    }
  }
  if constexpr (TPR != 0) {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if constexpr (CODES) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
  } else {
    cta_reduce<CODES>(ss, top, red);
  }
  if (!live) return;
  const RowFactors f = RowFactors::of<CODES>(a, row, ss, top, t == 0);
  YT *yr = static_cast<YT *>(a.y) + row * a.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t + i * tpr;
    if (c < nv) {
      const int lo = lo_of(c);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= f.rstd;
      if (WAN_DBG_OK(yr + max(lo, 0), (min(lo + 8, D) - max(lo, 0)) * sizeof(YT), a.y,
                     static_cast<YT *>(a.y) + (a.rows - 1) * a.ldy + D, a.dbg, WAN_DBG_CODE_BASE + 14)) {
        if constexpr (CODES) {
          if (whole(c)) store8_codes(yr + lo, v[i], f.inv);
          else store_part_codes(yr, lo, D, v[i], f.inv);
        } else {
          if (whole(c)) store8(yr + lo, v[i]);
          else store_part(yr, lo, D, v[i]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- ragged rows
// Bytes [p, p + n) of global memory, in a shared buffer that holds byte p at
// offset (p % 16): whole 16-byte pieces where they lie inside the range, the
// two ends element by element (E bytes each).
template <typename T>
__device__ __forceinline__ void pieces_in(uint8_t *buf, const T *p, int n) {
  const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15), head = min(n, off ? (16 - off) / (int)sizeof(T) : 0);
  const int whole = (n - head) / (16 / (int)sizeof(T)), tail = n - head - whole * (16 / (int)sizeof(T));
  T *b = reinterpret_cast<T *>(buf + off);
  const uint4 *src = reinterpret_cast<const uint4 *>(p + head);
  uint4 *dst = reinterpret_cast<uint4 *>(b + head);
  for (int i = threadIdx.x; i < whole; i += blockDim.x) dst[i] = __ldcs(src + i);
  if (threadIdx.x < head) b[threadIdx.x] = p[threadIdx.x];
  if (threadIdx.x < tail) b[n - tail + threadIdx.x] = p[n - tail + threadIdx.x];
}
template <typename T>
__device__ __forceinline__ void pieces_out(T *p, const uint8_t *buf, int n) {
  const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15), head = min(n, off ? (16 - off) / (int)sizeof(T) : 0);
  const int whole = (n - head) / (16 / (int)sizeof(T)), tail = n - head - whole * (16 / (int)sizeof(T));
  const T *b = reinterpret_cast<const T *>(buf + off);
  uint4 *dst = reinterpret_cast<uint4 *>(p + head);
  const uint4 *src = reinterpret_cast<const uint4 *>(b + head);
  for (int i = threadIdx.x; i < whole; i += blockDim.x) __stcs(dst + i, src[i]);
  if (threadIdx.x < head) p[threadIdx.x] = b[threadIdx.x];
  if (threadIdx.x < tail) p[n - tail + threadIdx.x] = b[n - tail + threadIdx.x];
}

constexpr int RAGGED_NV = 16;                              // most elements of a thread
constexpr int RAGGED_CTA = RMS_MAX_D / RAGGED_NV;
constexpr int RAGGED_SHORT_D = 4096;                       // widest row that takes 8 elements a thread

// One CTA per row, NV elements a thread (every blockDim-th). Two buffers: x in,
// then y out; r in, then h out.
template <typename XT, typename RT, bool RES, typename YT, int NV>
__global__ void __launch_bounds__(RAGGED_CTA) rmsnorm_ragged_kernel(const RmsArgs a, int buf_bytes) {
  constexpr bool CODES = sizeof(YT) == 1;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2][32];
  uint8_t *xb = smem, *rb = smem + buf_bytes;
  const long long row = blockIdx.x;
  const int D = a.D;
  const XT *xr = static_cast<const XT *>(a.x) + row * a.ldx;
  const RT *rr = RES ? static_cast<const RT *>(a.r) + row * a.ldr : nullptr;
  pieces_in(xb, xr, D);
  if constexpr (RES) pieces_in(rb, rr, D);
  __syncthreads();
  const XT *xs = reinterpret_cast<const XT *>(xb + (reinterpret_cast<uintptr_t>(xr) & 15));
  const RT *rs = reinterpret_cast<const RT *>(rb + (reinterpret_cast<uintptr_t>(rr) & 15));
  float h[NV], g[NV];
  float ss = 0.f, top = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    g[i] = a.g && c < D ? __ldg(a.g + c) : 1.f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    h[i] = 0.f;
    if (c < D) {
      h[i] = ElemIO<XT>::load(xs + c);
      if constexpr (RES) h[i] += ElemIO<RT>::load(rs + c);
      ss = fmaf(h[i], h[i], ss);
      if constexpr (CODES) top = fmaxf(top, fabsf(h[i] * g[i]));
    }
  }
  cta_reduce<CODES>(ss, top, red);                         // its barrier: both buffers have been read
  const RowFactors f = RowFactors::of<CODES>(a, row, ss, top, threadIdx.x == 0);
  YT *yr = static_cast<YT *>(a.y) + row * a.ldy;
  RT *hr = RES && a.h ? static_cast<RT *>(a.h) + row * a.ldh : nullptr;
  YT *ys = reinterpret_cast<YT *>(xb + (reinterpret_cast<uintptr_t>(yr) & 15));
  RT *hs = reinterpret_cast<RT *>(rb + (reinterpret_cast<uintptr_t>(hr) & 15));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < D) {
      if (RES && hr) ElemIO<RT>::store(hs + c, h[i]);
      const float y = h[i] * g[i] * f.rstd;
      if constexpr (CODES) ys[c] = __nv_cvt_float_to_fp8(__fmul_rn(y, f.inv), __NV_SATFINITE, __NV_E4M3);
      else ElemIO<YT>::store(ys + c, y);
    }
  }
  __syncthreads();
  if (WAN_DBG_OK(yr, D * sizeof(YT), a.y, static_cast<YT *>(a.y) + (a.rows - 1) * a.ldy + D, a.dbg, WAN_DBG_CODE_BASE + 14))
    pieces_out(yr, xb, D);
  if constexpr (RES) {
    if (hr && WAN_DBG_OK(hr, D * sizeof(RT), a.h, static_cast<RT *>(a.h) + (a.rows - 1) * a.ldh + D, a.dbg, WAN_DBG_CODE_BASE + 12))
      pieces_out(hr, rb, D);
  }
}

// ---------------------------------------------------------------- launches
enum RowLayout { ROWS_ALIGNED, ROWS_SHIFTED, ROWS_RAGGED };

template <typename XT, typename RT, bool RES, typename YT, int NV, int TPR>
int rms_launch(const RmsArgs &a, RowLayout lay, int threads, cudaStream_t s) {
  const int per = TPR ? threads / TPR : 1;
  const long long grid = ((long long)a.rows + per - 1) / per;
  if constexpr (TPR || NV > 1) {               // one group a thread, a CTA to a row: shifted rows only
    if (lay == ROWS_ALIGNED) {
      rmsnorm_kernel<XT, RT, RES, YT, NV, TPR, false><<<(unsigned)grid, threads, 0, s>>>(a);
      WAN_CHECK_LAUNCH("rmsnorm");
      return WAN_OK;
    }
  }
  rmsnorm_kernel<XT, RT, RES, YT, NV, TPR, true><<<(unsigned)grid, threads, 0, s>>>(a);
  WAN_CHECK_LAUNCH("rmsnorm");
  return WAN_OK;
}

// Shared memory of a ragged row of D elements: each buffer with 16 bytes for the
// row's offset in them.
constexpr int ragged_buf(int D, int es) { return (D * es + 16 + 15) / 16 * 16; }

// The long form may take more than the 48 KB (with its own 256 bytes) that a
// kernel gets unasked. The limit belongs to the kernel and not to the call, so it
// is raised once on a device, to what the widest row takes: raised to each call's
// own size, it could be lowered by one host thread before another one's launch.
template <typename XT, typename RT, bool RES, typename YT, int NV>
int rms_launch_ragged(const RmsArgs &a, int threads, cudaStream_t s) {
  constexpr int es = sizeof(XT) > sizeof(YT) ? sizeof(XT) : sizeof(YT);
  constexpr int widest = NV == RAGGED_NV ? RMS_MAX_D : RAGGED_SHORT_D;
  constexpr int most = ragged_buf(widest, es) + (RES ? ragged_buf(widest, sizeof(RT)) : 0);
  if constexpr (most > 48 * 1024 - 256) {
    static std::atomic<uint64_t> ready{0};       // devices whose limit is raised
    int dev = 0;
    WAN_TRY_CUDA(cudaGetDevice(&dev), "rmsnorm device");
    if (dev >= 64 || !(ready.load() >> dev & 1)) {
      WAN_TRY_CUDA(cudaFuncSetAttribute(rmsnorm_ragged_kernel<XT, RT, RES, YT, NV>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, most), "rmsnorm smem attribute");
      if (dev < 64) ready.fetch_or(uint64_t(1) << dev);
    }
  }
  const int xb = ragged_buf(a.D, es), rb = RES ? ragged_buf(a.D, sizeof(RT)) : 0;
  rmsnorm_ragged_kernel<XT, RT, RES, YT, NV><<<(unsigned)a.rows, threads, xb + rb, s>>>(a, xb);
  WAN_CHECK_LAUNCH("rmsnorm");
  return WAN_OK;
}

// Groups per thread, measured: a warp or part of one holds up to 64 groups; then
// two a thread (20000 x 1000 f32: 26.7 us, 28.7 with one; 20000 x 777 shifted
// bf16 29.4, 33.1), but one for shifted rows of up to 96 groups (20000 x 603
// onto codes: 32.4 us, 38.7 with two), and four where two would take more than
// 512 threads.
template <typename XT, typename RT, bool RES, typename YT>
int rms_shape(const RmsArgs &a, RowLayout lay, cudaStream_t s) {
  const int n = lay == ROWS_RAGGED ? a.D : (a.D + (lay == ROWS_SHIFTED ? 14 : 0)) / 8;   // groups of any row, at most
  auto threads = [&](int per) { return ((n + per - 1) / per + 31) / 32 * 32; };
  if (lay != ROWS_RAGGED) {
    if (n <= 8) return rms_launch<XT, RT, RES, YT, 1, 8>(a, lay, ROW_CTA, s);
    if (n <= 16) return rms_launch<XT, RT, RES, YT, 1, 16>(a, lay, ROW_CTA, s);
    if (n <= 32) return rms_launch<XT, RT, RES, YT, 1, 32>(a, lay, ROW_CTA, s);
    if (n <= 64) return rms_launch<XT, RT, RES, YT, 2, 32>(a, lay, ROW_CTA, s);
    if (n <= 96 && lay == ROWS_SHIFTED) return rms_launch<XT, RT, RES, YT, 1, 0>(a, lay, threads(1), s);
    if (n <= 1024) return rms_launch<XT, RT, RES, YT, 2, 0>(a, lay, threads(2), s);
    return rms_launch<XT, RT, RES, YT, 4, 0>(a, lay, threads(4), s);
  }
  if (n <= RAGGED_SHORT_D) return rms_launch_ragged<XT, RT, RES, YT, 8>(a, threads(8), s);
  return rms_launch_ragged<XT, RT, RES, YT, RAGGED_NV>(a, threads(RAGGED_NV), s);
}

template <typename XT, typename YT>
int rms_res(const RmsArgs &a, int res_dtype, RowLayout lay, cudaStream_t s) {
  if (!a.r) return rms_shape<XT, float, false, YT>(a, lay, s);
  if (res_dtype == WAN_BF16) return rms_shape<XT, __nv_bfloat16, true, YT>(a, lay, s);
  return rms_shape<XT, float, true, YT>(a, lay, s);
}

template <typename XT>
int rms_out(const RmsArgs &a, int res_dtype, int y_dtype, RowLayout lay, cudaStream_t s) {
  if (y_dtype == WAN_FP8) return rms_res<XT, uint8_t>(a, res_dtype, lay, s);
  if (y_dtype == WAN_BF16) return rms_res<XT, __nv_bfloat16>(a, res_dtype, lay, s);
  return rms_res<XT, float>(a, res_dtype, lay, s);
}

}  // namespace

int launch_rmsnorm(int rows, int D, const void *x, int x_dtype, long long ldx, const void *r, int res_dtype,
                   long long ldr, const float *g, float eps, void *h, long long ldh, void *y, int y_dtype,
                   long long ldy, float *scale, cudaStream_t s) {
  const long long least = r && ldr < ldx ? ldr : ldx;
  const int inner = rows == 1 || least < 1 ? 0 : rows - (int)((7 + least - 1) / least);
  RmsArgs a = {rows, D, x, ldx, r, ldr, g, eps, h, ldh, y, ldy, scale, inner, dbg_word()};
  // a matrix that is not there goes along with x, a single row with itself
  auto mod8 = [&](const void *p, long long ld) { return (int)((rows == 1 ? 0 : p ? ld : ldx) & 7); };
  const int m = mod8(x, ldx);
  RowLayout lay = ROWS_RAGGED;
  if (mod8(r, ldr) == m && mod8(h, ldh) == m && mod8(y, ldy) == m) {
    if (D % 8 == 0 && m == 0) lay = ROWS_ALIGNED;
    else if ((D + 14) / 8 <= 4 * VEC_CTA) lay = ROWS_SHIFTED;
  }
  return x_dtype == WAN_BF16 ? rms_out<__nv_bfloat16>(a, res_dtype, y_dtype, lay, s)
                             : rms_out<float>(a, res_dtype, y_dtype, lay, s);
}

}  // namespace wan

// Row RMS norm with the residual's addition (wan_rmsnorm):
//
//     h = x + r                       (h = x without a residual)
//     y = (h g) rstd,  rstd = 1 / sqrt(sum h^2 / D + eps)
//
// stored as bf16 / float32, or as e4m3 codes with one scale per row. x, r, h
// and y cross HBM once: a row stays in registers between its reads and its
// writes, so the kernel is bound by those bytes alone.
//
// The sum of squares and the row's maximum are reduced together: rounding is
// monotone, so max |(h g) rstd| = fl(max |h g| * rstd) exactly, and the scale
// of the e4m3 output needs no second pass after rstd is known. h is the
// float32 sum, rounded only where it is stored (the norm sees the unrounded
// sum: one rounding less than adding, storing and reading back).
#include "common.cuh"
#include "e4m3.cuh"

#include <float.h>

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
  int *dbg;
};

// V consecutive elements at p as floats (V = 8: the caller checked alignment).
template <int V>
__device__ __forceinline__ void ld_vec(const float *p, float (&v)[V]) {
  if constexpr (V == 8) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = p[e];
  }
}
template <int V>
__device__ __forceinline__ void ld_vec(const __nv_bfloat16 *p, float (&v)[V]) {
  if constexpr (V == 8) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = __bfloat162float(p[e]);
  }
}
template <int V>
__device__ __forceinline__ void st_vec(float *p, const float (&v)[V]) {
  if constexpr (V == 8) {
    store4(p, make_float4(v[0], v[1], v[2], v[3]));
    store4(p + 4, make_float4(v[4], v[5], v[6], v[7]));
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) p[e] = v[e];
  }
}
template <int V>
__device__ __forceinline__ void st_vec(__nv_bfloat16 *p, const float (&v)[V]) {
  if constexpr (V == 8) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) p[e] = __float2bfloat16_rn(v[e]);
  }
}
// e4m3 codes of v * inv
template <int V>
__device__ __forceinline__ void st_codes(uint8_t *p, const float (&v)[V], float inv) {
  if constexpr (V == 8) {
    uint2 o;
    o.x = quant4(make_float4(v[0], v[1], v[2], v[3]), inv);
    o.y = quant4(make_float4(v[4], v[5], v[6], v[7]), inv);
    *reinterpret_cast<uint2 *>(p) = o;
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) p[e] = __nv_cvt_float_to_fp8(__fmul_rn(v[e], inv), __NV_SATFINITE, __NV_E4M3);
  }
}

// TPR threads of one warp per row (several rows per CTA), or TPR = 0: the
// whole CTA per row. NV vectors of V elements per thread. RES: 0 none, else
// RT is the residual's type.
template <typename XT, typename RT, bool RES, typename YT, int V, int NV, int TPR>
__global__ void rmsnorm_kernel(const RmsArgs a) {
  constexpr bool CODES = sizeof(YT) == 1;
  __shared__ float red[2][32];
  const int tpr = TPR ? TPR : blockDim.x;
  const int t = TPR ? (int)(threadIdx.x % TPR) : (int)threadIdx.x;
  const long long row = TPR ? (long long)blockIdx.x * (blockDim.x / TPR) + threadIdx.x / TPR : blockIdx.x;
  const bool live = row < a.rows;
  const int nv = a.D / V;
  float v[NV][V];
  float ss = 0.f, top = 0.f;
  if (live) {
    const XT *xr = static_cast<const XT *>(a.x) + row * a.ldx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * tpr;
      if (c < nv) ld_vec<V>(xr + (long long)c * V, v[i]);
    }
    if constexpr (RES) {
      const RT *rr = static_cast<const RT *>(a.r) + row * a.ldr;
      float q[NV][V];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * tpr;
        if (c < nv) ld_vec<V>(rr + (long long)c * V, q[i]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * tpr;
        if (c < nv) {
#pragma unroll
          for (int e = 0; e < V; ++e) v[i][e] += q[i][e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * tpr;
      if (c < nv) {
        if constexpr (RES) {
          if (a.h) {
            RT *hp = static_cast<RT *>(a.h) + row * a.ldh + (long long)c * V;
            if (WAN_DBG_OK(hp, V * sizeof(RT), a.h, static_cast<RT *>(a.h) + (a.rows - 1) * a.ldh + a.D, a.dbg,
                           WAN_DBG_CODE_BASE + 12))
              st_vec<V>(hp, v[i]);
          }
        }
#pragma unroll
        for (int e = 0; e < V; ++e) ss = fmaf(v[i][e], v[i][e], ss);
        if (a.g) {
#pragma unroll
          for (int e = 0; e < V; e += 4) {
            if constexpr (V == 8) {
              const float4 gv = load4(a.g + c * V + e);
              v[i][e] *= gv.x; v[i][e + 1] *= gv.y; v[i][e + 2] *= gv.z; v[i][e + 3] *= gv.w;
            } else {
              v[i][e] *= a.g[c];
            }
          }
        }
        if constexpr (CODES) {
#pragma unroll
          for (int e = 0; e < V; ++e) top = fmaxf(top, fabsf(v[i][e]));
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
  if (!live) return;
  const float rstd = 1.0f / sqrtf(ss / (float)a.D + a.eps);
  float inv = 1.f;
  if constexpr (CODES) {
    const float amax = top * rstd;
    inv = fminf(e4m3_inv_scale(amax), FLT_MAX);     // amax below 448 / FLT_MAX: no infinite factor
    if (!(amax == amax)) inv = amax;                // a row with NaN: every code NaN
    if (t == 0 && WAN_DBG_OK(a.scale + row, 4, a.scale, a.scale + a.rows, a.dbg, WAN_DBG_CODE_BASE + 13))
      a.scale[row] = __fdiv_rn(amax, E4M3_MAX);
  }
  YT *yr = static_cast<YT *>(a.y) + row * a.ldy;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t + i * tpr;
    if (c < nv) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] *= rstd;
      YT *yp = yr + (long long)c * V;
      if (WAN_DBG_OK(yp, V * sizeof(YT), a.y, static_cast<YT *>(a.y) + (a.rows - 1) * a.ldy + a.D, a.dbg,
                     WAN_DBG_CODE_BASE + 14)) {
        if constexpr (CODES) st_codes<V>(yp, v[i], inv);
        else st_vec<V>(yp, v[i]);
      }
    }
  }
}

constexpr int ROW_CTA = 128;          // threads of a CTA that holds several rows

template <typename XT, typename RT, bool RES, typename YT, int V, int NV, int TPR>
int rms_launch(const RmsArgs &a, int threads, cudaStream_t s) {
  const int per = TPR ? threads / TPR : 1;
  const long long grid = ((long long)a.rows + per - 1) / per;
  rmsnorm_kernel<XT, RT, RES, YT, V, NV, TPR><<<(unsigned)grid, threads, 0, s>>>(a);
  WAN_CHECK_LAUNCH("rmsnorm");
  return WAN_OK;
}

template <typename XT, typename RT, bool RES, typename YT>
int rms_shape(const RmsArgs &a, bool vec, cudaStream_t s) {
  const int nv = vec ? a.D / 8 : a.D;
  if (vec) {
    if (nv <= 8) return rms_launch<XT, RT, RES, YT, 8, 1, 8>(a, ROW_CTA, s);
    if (nv <= 16) return rms_launch<XT, RT, RES, YT, 8, 1, 16>(a, ROW_CTA, s);
    if (nv <= 32) return rms_launch<XT, RT, RES, YT, 8, 1, 32>(a, ROW_CTA, s);
    if (nv <= 64) return rms_launch<XT, RT, RES, YT, 8, 2, 32>(a, ROW_CTA, s);
    auto threads = [&](int per) { return ((nv + per - 1) / per + 31) / 32 * 32; };
    if (nv <= 256) return rms_launch<XT, RT, RES, YT, 8, 1, 0>(a, threads(1), s);
    if (nv <= 1024) return rms_launch<XT, RT, RES, YT, 8, 2, 0>(a, threads(2), s);
    return rms_launch<XT, RT, RES, YT, 8, 4, 0>(a, threads(4), s);
  }
  auto threads = [&](int per) { return ((nv + per - 1) / per + 31) / 32 * 32; };
  if (nv <= 128) return rms_launch<XT, RT, RES, YT, 1, 4, 32>(a, ROW_CTA, s);
  if (nv <= 2048) return rms_launch<XT, RT, RES, YT, 1, 8, 0>(a, threads(8), s);
  return rms_launch<XT, RT, RES, YT, 1, 32, 0>(a, threads(32), s);
}

template <typename XT, typename YT>
int rms_res(const RmsArgs &a, int res_dtype, bool vec, cudaStream_t s) {
  if (!a.r) return rms_shape<XT, float, false, YT>(a, vec, s);
  if (res_dtype == WAN_BF16) return rms_shape<XT, __nv_bfloat16, true, YT>(a, vec, s);
  return rms_shape<XT, float, true, YT>(a, vec, s);
}

template <typename XT>
int rms_out(const RmsArgs &a, int res_dtype, int y_dtype, bool vec, cudaStream_t s) {
  if (y_dtype == WAN_FP8) return rms_res<XT, uint8_t>(a, res_dtype, vec, s);
  if (y_dtype == WAN_BF16) return rms_res<XT, __nv_bfloat16>(a, res_dtype, vec, s);
  return rms_res<XT, float>(a, res_dtype, vec, s);
}

}  // namespace

int launch_rmsnorm(int rows, int D, const void *x, int x_dtype, long long ldx, const void *r, int res_dtype,
                   long long ldr, const float *g, float eps, void *h, long long ldh, void *y, int y_dtype,
                   long long ldy, float *scale, cudaStream_t s) {
  RmsArgs a = {rows, D, x, ldx, r, ldr, g, eps, h, ldh, y, ldy, scale, dbg_word()};
  // 8 elements a thread at a time where every row starts on a 16-byte (codes:
  // 8-byte) boundary, else one by one
  const bool vec = D % 8 == 0 && (rows == 1 || (ldx % 8 == 0 && (!r || ldr % 8 == 0) && (!h || ldh % 8 == 0) && ldy % 8 == 0));
  return x_dtype == WAN_BF16 ? rms_out<__nv_bfloat16>(a, res_dtype, y_dtype, vec, s)
                             : rms_out<float>(a, res_dtype, y_dtype, vec, s);
}

}  // namespace wan

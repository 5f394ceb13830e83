// The epilogue of wan_linear, shared by its kernels. Internal header.
#pragma once

#include "common.cuh"

namespace wan {

// Arguments of a linear layer call (wan.h, wan_linear); strides in elements.
struct LinArgs {
  int M, N, K, fp8;
  const void *a; long long lda; const float *a_scale;
  const void *w; long long ldw; const float *w_scale; int w_scale_rows;   // w_scale_rows: one per weight row
  const void *bias;                                                       // bf16 [N] or NULL
  int act;                                                                // WAN_ACT_*
  const void *res; int res_f32; long long ldr;
  void *out; int out_f32; long long ldo;
};
int launch_linear(const LinArgs &g, cudaStream_t s);

struct LinEpilogue {
  const float *a_scale, *w_scale; int w_scale_rows;
  const __nv_bfloat16 *bias;
  int act;
  const void *res; long long ldr; int res_f32;
  void *out; long long ldo; int out_f32;
  int vec;                                  // rows of out and res hold aligned groups of 4 columns
  const void *out_hi; int *dbg;             // debug bounds checks: end of out
};

inline LinEpilogue lin_epilogue(const LinArgs &g) {
  LinEpilogue e = {};
  e.a_scale = g.a_scale; e.w_scale = g.w_scale; e.w_scale_rows = g.w_scale_rows;
  e.bias = static_cast<const __nv_bfloat16 *>(g.bias);
  e.act = g.act;
  e.res = g.res; e.ldr = g.ldr; e.res_f32 = g.res_f32;
  e.out = g.out; e.ldo = g.ldo; e.out_f32 = g.out_f32;
  e.vec = g.M == 1 || (g.ldo % 4 == 0 && (!g.res || g.ldr % 4 == 0));
  e.out_hi = static_cast<char *>(g.out) + ((g.M - 1) * g.ldo + g.N) * (g.out_f32 ? 4 : 2);
  e.dbg = dbg_word();
  return e;
}

// z / (1 + exp(-u)): the sigmoid form keeps the relative error of the tails,
// where 1 + tanh cancels. SiLU is u = z; the tanh form of GELU is
// 0.5 z (1 + tanh v) = z / (1 + exp(-2 v)), v = sqrt(2/pi) (z + 0.044715 z^3).
__device__ __forceinline__ float lin_gated(float z, float u) { return __fdividef(z, 1.0f + __expf(-u)); }

__device__ __forceinline__ float lin_act(float z, int act) {
  switch (act) {
    case WAN_ACT_GELU_TANH: {
      const float k0 = 2.0f * 0.7978845608028654f;
      return lin_gated(z, k0 * fmaf(0.044715f * z * z, z, z));
    }
    case WAN_ACT_SILU: return lin_gated(z, z);
    case WAN_ACT_RELU: return z < 0.f ? 0.f : z;      // NaN stays NaN
    default: return z;
  }
}

// Per-column operands of 4 columns n .. n + 3 (those below N).
struct LinColumns {
  float b[4], s[4];
  __device__ __forceinline__ void load(const LinEpilogue &e, int n, int N, bool f8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) { b[j] = 0.f; s[j] = 1.f; }
    if (n + 4 <= N) {
      if (e.bias) {
        const float4 v = load4(e.bias + n);
        b[0] = v.x; b[1] = v.y; b[2] = v.z; b[3] = v.w;
      }
      if (f8 && e.w_scale_rows) {
        const float4 v = load4(e.w_scale + n);
        s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (n + j < N) {
          if (e.bias) b[j] = __bfloat162float(e.bias[n + j]);
          if (f8 && e.w_scale_rows) s[j] = e.w_scale[n + j];
        }
      }
    }
    if (f8 && !e.w_scale_rows) {
      const float v = e.w_scale[0];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = v;
    }
  }
};

// Row m, columns n .. n + 3 (those below N) of the output from their sums.
__device__ __forceinline__ void lin_store4(const LinEpilogue &e, const LinColumns &c, int m, int n, int N, float4 acc,
                                           bool f8) {
  float v[4] = {acc.x, acc.y, acc.z, acc.w};
  const float as = f8 ? e.a_scale[m] : 1.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = lin_act(f8 ? fmaf(v[j], as * c.s[j], c.b[j]) : v[j] + c.b[j], e.act);
  const long long ro = (long long)m * e.ldr + n, oo = (long long)m * e.ldo + n;
  const float *rf = static_cast<const float *>(e.res);
  const __nv_bfloat16 *rh = static_cast<const __nv_bfloat16 *>(e.res);
  float *of = static_cast<float *>(e.out);
  __nv_bfloat16 *oh = static_cast<__nv_bfloat16 *>(e.out);
  if (e.vec && n + 4 <= N) {
    if (e.res) {
      const float4 r = e.res_f32 ? load4(rf + ro) : load4(rh + ro);
      v[0] += r.x; v[1] += r.y; v[2] += r.z; v[3] += r.w;
    }
    const float4 o = make_float4(v[0], v[1], v[2], v[3]);
    if (e.out_f32) {
      if (WAN_DBG_OK(of + oo, 16, e.out, e.out_hi, e.dbg, WAN_DBG_CODE_BASE + 15)) store4(of + oo, o);
    } else {
      if (WAN_DBG_OK(oh + oo, 8, e.out, e.out_hi, e.dbg, WAN_DBG_CODE_BASE + 15)) store4(oh + oo, o);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (n + j >= N) break;
    if (e.res) v[j] += e.res_f32 ? rf[ro + j] : __bfloat162float(rh[ro + j]);
    if (e.out_f32) {
      if (WAN_DBG_OK(of + oo + j, 4, e.out, e.out_hi, e.dbg, WAN_DBG_CODE_BASE + 15)) of[oo + j] = v[j];
    } else {
      if (WAN_DBG_OK(oh + oo + j, 2, e.out, e.out_hi, e.dbg, WAN_DBG_CODE_BASE + 15)) oh[oo + j] = __float2bfloat16_rn(v[j]);
    }
  }
}

}  // namespace wan

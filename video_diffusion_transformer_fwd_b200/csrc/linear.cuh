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
int gemm_tc_linear(const LinArgs &g, int bn, cudaStream_t s);   // CTA pairs (gemm_tc.cu)

// The tensor core rounds its running sum of bf16 products toward zero, an error
// that grows with the number of steps (relative 1.1e-9 K, measured against 64
// bits). Under a bf16 output that is nothing, but a float32 output gets an
// accumulator for every 12 steps of 64, and these are added in float32. On CTA
// pairs only from 33 steps on: one accumulator is off by 2.2e-6 at K = 2048, and
// parts need narrower tiles (4096 x 4096 x 2048 onto float32: 61 us with one, 72
// in parts; x 4096: 117 with two of 32 steps, 119 in parts). e4m3 products need
// none (4.9e-7 at K = 13824).
constexpr int LIN_PART_STEPS = 12;
inline int lin_parts(const LinArgs &g, int steps) {
  return g.fp8 || !g.out_f32 ? 1 : (steps + LIN_PART_STEPS - 1) / LIN_PART_STEPS;
}
inline int lin_pair_parts(const LinArgs &g, int steps) { return steps <= 32 ? 1 : lin_parts(g, steps); }
constexpr int LIN_PARTS_BN = 160;         // widest pair tile with several parts: 3 x 160 of TMEM's 512 columns

struct LinEpilogue {
  const float *a_scale, *w_scale; int w_scale_rows;
  const __nv_bfloat16 *bias;
  int act;
  const void *res; long long ldr; int res_f32;
  void *out; long long ldo; int out_f32;
  int vec_out, vec_res;                     // every row of out (res) starts on a 16-byte boundary
  const void *out_hi; int *dbg;             // debug bounds checks: end of out
};

inline LinEpilogue lin_epilogue(const LinArgs &g) {
  LinEpilogue e = {};
  e.a_scale = g.a_scale; e.w_scale = g.w_scale; e.w_scale_rows = g.w_scale_rows;
  e.bias = static_cast<const __nv_bfloat16 *>(g.bias);
  e.act = g.act;
  e.res = g.res; e.ldr = g.ldr; e.res_f32 = g.res_f32;
  e.out = g.out; e.ldo = g.ldo; e.out_f32 = g.out_f32;
  e.vec_out = g.ldo % (g.out_f32 ? 4 : 8) == 0;
  e.vec_res = !g.res || g.ldr % (g.res_f32 ? 4 : 8) == 0;
  e.out_hi = static_cast<char *>(g.out) + ((g.M - 1) * g.ldo + g.N) * (g.out_f32 ? 4 : 2);
  e.dbg = dbg_word();
  return e;
}

// z / (1 + 2^x): the sigmoid form has no cancellation in the tails, as 1 + tanh
// has, and takes two steps of the special-function unit (2^x and the reciprocal,
// each within 2^-22). The error is relative to the result and grows with the
// exponent, whose own rounding counts |x| times: (6 + 2.2 |x|) 2^-23 at most, below
// a bf16 output's half step throughout. Where 1 + 2^x passes 2^126 the quotient is
// flushed to 0 (|result| < 1.1e-36). SiLU is x = -z log2(e); the tanh form of
// GELU is 0.5 z (1 + tanh v) = z / (1 + exp(-2 v)), v = sqrt(2/pi) (z + 0.044715 z^3).
__device__ __forceinline__ float lin_gated(float z, float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return z * r;
}

__device__ __forceinline__ float lin_act(float z, int act) {
  constexpr float log2e = 1.4426950408889634f;
  switch (act) {
    case WAN_ACT_GELU_TANH: {
      constexpr float c0 = -2.0f * 0.7978845608028654f * log2e, c1 = c0 * 0.044715f;
      return lin_gated(z, z * fmaf(z * z, c1, c0));
    }
    case WAN_ACT_SILU: return lin_gated(z, -log2e * z);
    case WAN_ACT_RELU: return z < 0.f ? 0.f : z;      // NaN stays NaN
    default: return z;
  }
}

// The same on several values, the choice outside the loop.
template <int C>
__device__ __forceinline__ void lin_act_row(float (&v)[C], int act) {
  if (act == WAN_ACT_GELU_TANH) {
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = lin_act(v[j], WAN_ACT_GELU_TANH);
  } else if (act == WAN_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = lin_act(v[j], WAN_ACT_SILU);
  } else if (act == WAN_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = lin_act(v[j], WAN_ACT_RELU);
  }
}

__device__ __forceinline__ void lin_put(const LinEpilogue &e, int m, int n, float v) {
  const long long o = (long long)m * e.ldo + n;
  if (e.out_f32) {
    float *p = static_cast<float *>(e.out) + o;
    if (WAN_DBG_OK(p, 4, e.out, e.out_hi, e.dbg, WAN_DBG_CODE_BASE + 15)) *p = v;
  } else {
    __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(e.out) + o;
    if (WAN_DBG_OK(p, 2, e.out, e.out_hi, e.dbg, WAN_DBG_CODE_BASE + 15)) *p = __float2bfloat16_rn(v);
  }
}
}  // namespace wan

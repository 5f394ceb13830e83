// e4m3 conversion shared by the quantizing kernels: a row's scale is
// amax / 448 and an element's code is the e4m3 value nearest to
// x * (448 / amax), ties to even, clamped to +-448. Internal header.
#pragma once

#include "common.cuh"

#include <cuda_fp8.h>

namespace wan {

constexpr float E4M3_MAX = 448.f;

// four values -> four e4m3 bytes, the first in the lowest byte
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ float e4m3_inv_scale(float amax) {
  return amax > 0.f ? __fdiv_rn(E4M3_MAX, amax) : 0.f;
}

__device__ __forceinline__ float absmax4(float4 v) {
  return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

__device__ __forceinline__ uint32_t quant4(float4 v, float inv) {
  return e4m3x4(__fmul_rn(v.x, inv), __fmul_rn(v.y, inv), __fmul_rn(v.z, inv), __fmul_rn(v.w, inv));
}

}  // namespace wan

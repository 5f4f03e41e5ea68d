// Roots and reciprocals from the hardware's approximations and one Newton step
// with a fused residual (Markstein).  tests/test_gpu_roots.py compares them with
// the correctly rounded ones on every float32 of the ranges given here.
#pragma once

#include "pairs.cuh"

namespace moe {

__device__ __forceinline__ float approx_rsqrt(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  return y;
}
// 1 / x within 2 u, x from 2^-126 to 2^126
__device__ __forceinline__ float approx_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// sqrt(v) rounded to nearest, v from 2^-102 (below, the residual underflows) to
// the largest finite
__device__ __forceinline__ float2 root2(float2 v) {
  const float2 y = make_float2(approx_rsqrt(v.x), approx_rsqrt(v.y));
  const float2 s = mul2(v, y);
  return fma2(fma2(mul2(s, both(-1.f)), s, v), mul2(y, both(0.5f)), s);
}
// 1 / x rounded to nearest, x from 2^-126 to 2^126
__device__ __forceinline__ float reciprocal(float x) {
  const float y = approx_rcp(x);
  return fmaf(fmaf(-x, y, 1.f), y, y);
}
// 1 / sqrt(v) within 2 u, v from 2^-126 on
__device__ __forceinline__ float rsqrt_of(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.f);
  return v > 0.f && v < INFINITY ? fmaf(0.5f * r, e, r) : r;
}

}  // namespace moe

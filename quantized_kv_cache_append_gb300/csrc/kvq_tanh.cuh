// kvq_tanh.cuh -- tanh of a score, for the attention kernels that cap them.
//
// Up to |y| = 0.625 it is y P(y^2), P of degree 5 fitted to tanh(y) / y there
// (weighted least squares on Chebyshev nodes, relative error 4e-9; evaluated
// in fp32 within two half steps); above, 1 - 2 / (1 + e^(2|y|)), where the
// cancellation costs at most one bit.  Scores mostly stay below the cap's
// half, so a warp whose scores are all small takes only the first form: 7
// FMA-pipe instructions and no special function.
#pragma once

#include "kvq_ptx.cuh"

namespace kvq {

constexpr float kTanhSmall = 0.625f;

static __device__ __forceinline__ float tanh_small(float y) {
  const float x = y * y;
  float p = fmaf(-0.00565999f, x, 0.020590989f);
  p = fmaf(p, x, -0.053721067f);
  p = fmaf(p, x, 0.13331127f);
  p = fmaf(p, x, -0.3333326f);
  return fmaf(y * x, p, y);
}

// any y; NaN stays NaN, infinities give +-1
static __device__ __forceinline__ float tanh_any(float y) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + fast_exp2(2.8853900817779268f * fabsf(y))));
  return fabsf(y) > kTanhSmall ? copysignf(fmaf(-2.0f, r, 1.0f), y) : tanh_small(y);
}

}  // namespace kvq

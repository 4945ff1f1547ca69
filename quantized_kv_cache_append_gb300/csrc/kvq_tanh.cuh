// kvq_tanh.cuh -- capped scores of the decode: cap * tanh(z / cap).
//
// Up to |y| = |z / cap| = 0.625 it is z + z x P(x), x = y^2, P of degree 4 from a
// polynomial of degree 5 fitted to tanh(y) / y there (weighted least squares on
// Chebyshev nodes; relative error 1.1e-8 with the coefficients as fp32 holds them,
// a sixth of an fp32 half step); above, cap (1 - 2 / (1 + e^(2|y|))), where
// the cancellation costs at most one bit.  Scores mostly stay below the cap's
// half, so a warp whose scores are all small takes only the first form, two
// scores an instruction: 8 packed instructions and no special function.
#pragma once

#include "kvq_ptx.cuh"
#include "kvq_tc.cuh"

namespace kvq {

constexpr float kTanhSmall = 0.625f;

static __device__ __forceinline__ void cap_small(float& z0, float& z1, float cap_inv) {
  float x0, x1, p0, p1;
  mul_f32x2(x0, x1, z0, z1, cap_inv, cap_inv);
  mul_f32x2(x0, x1, x0, x1, x0, x1);
  fma_f32x2(p0, p1, x0, x1, -0.00565999f, -0.00565999f, 0.020590989f, 0.020590989f);
  fma_f32x2(p0, p1, p0, p1, x0, x1, -0.053721067f, -0.053721067f);
  fma_f32x2(p0, p1, p0, p1, x0, x1, 0.13331127f, 0.13331127f);
  fma_f32x2(p0, p1, p0, p1, x0, x1, -0.3333326f, -0.3333326f);
  mul_f32x2(p0, p1, p0, p1, x0, x1);
  fma_f32x2(z0, z1, z0, z1, p0, p1, z0, z1);
}

// any z (small: cap_small's result); NaN stays NaN, infinities give +-cap
static __device__ __forceinline__ float cap_any(float z, float small, float cap, float cap_inv) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + fast_exp2(2.8853900817779268f * cap_inv * fabsf(z))));
  return fabsf(z) > kTanhSmall * cap ? copysignf(fmaf(-2.0f * cap, r, cap), z) : small;
}

}  // namespace kvq

// Cap and distance bias of 32 scores of a row (or column), for the forward and
// backward kernels of the dense masked attention.
#pragma once

#include "sm100.cuh"

namespace vsa {
namespace masked {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;

// Per-row constants: `c` turns raw scores into log2 units, cap2 = cap log2(e),
// in = scale / cap, slope in log2 units.
struct ScoreTerms {
  float c, cap2, in, slope;
};

// Raw scores x (sums of products) -> log2 units, except that without cap and bias
// they stay raw (the caller's exponential applies c). With a cap t receives
// tanh(score / cap). Distance of column u: |d0 + dir u|, dir = 1 or -1.
//
// tanh: 1 - 2 / (1 + e^(2y)) takes two operations of the exponential unit per
// score, which then bounds the kernels. Where all of a warp's 32 x 32 scores have
// |y| <= 0.6 (a cap well above the scores, as caps are) it is y (1 + z p(z)),
// z = y^2, on the FMA pipe: p of degree 4, least squares with weights driven to
// equal extrema, relative error below 2^-23.
// Bias: where the columns lie on one side of every row of the warp, it is linear in
// the column: two operations for a pair of scores.
// Both together: 362 -> STREAMUS us for 2 x 1,111 queries over 5,003 keys, 24 heads.
template <bool kCap, bool kBias>
__device__ __forceinline__ void score_terms(float (&x)[32], float (&t)[32], const ScoreTerms& s, float d0, float dir) {
  uint64_t mul = pack_f32x2(s.c, s.c);          // what the bias step still multiplies by
  if constexpr (kCap) {
    float top = 0.0f;
#pragma unroll
    for (int u = 0; u < 32; ++u) top = fmaxf(top, fabsf(x[u]));
    const uint64_t in2 = pack_f32x2(s.in, s.in);
    if (__all_sync(0xffffffffu, top * s.in <= 0.6f)) {
      const uint64_t one = pack_f32x2(1.0f, 1.0f);
#pragma unroll
      for (int u = 0; u < 32; u += 2) {
        const uint64_t y = mul_f32x2(pack_f32x2(x[u], x[u + 1]), in2), z = mul_f32x2(y, y);
        uint64_t p = pack_f32x2(-0.00589513499f, -0.00589513499f);
        p = fma_f32x2(p, z, pack_f32x2(0.0207959544f, 0.0207959544f));
        p = fma_f32x2(p, z, pack_f32x2(-0.0537838265f, -0.0537838265f));
        p = fma_f32x2(p, z, pack_f32x2(0.133319244f, 0.133319244f));
        p = fma_f32x2(p, z, pack_f32x2(-0.333332986f, -0.333332986f));
        unpack_f32x2(mul_f32x2(y, fma_f32x2(p, z, one)), t[u], t[u + 1]);
      }
    } else {
      const float in_e = 2.0f * kLog2e * s.in;
#pragma unroll
      for (int u = 0; u < 32; ++u) t[u] = fmaf(-2.0f, rcp_approx(1.0f + ex2_approx(x[u] * in_e)), 1.0f);
    }
    mul = pack_f32x2(s.cap2, s.cap2);
  }
  float(&y)[32] = kCap ? t : x;
  if constexpr (kBias) {
    const float d31 = fmaf(dir, 31.0f, d0);
    const bool right = __all_sync(0xffffffffu, d0 >= 0.0f && d31 >= 0.0f);
    const bool left = __all_sync(0xffffffffu, d0 <= 0.0f && d31 <= 0.0f);
    if (right || left) {
      const float k = right ? -s.slope : s.slope, step = k * dir;
      const uint64_t base = pack_f32x2(k * d0, k * d0), step2 = pack_f32x2(step, step);
#pragma unroll
      for (int u = 0; u < 32; u += 2) {
        const uint64_t b = fma_f32x2(step2, pack_f32x2(static_cast<float>(u), static_cast<float>(u + 1)), base);
        unpack_f32x2(fma_f32x2(pack_f32x2(y[u], y[u + 1]), mul, b), x[u], x[u + 1]);
      }
    } else {
      const float m = kCap ? s.cap2 : s.c;
#pragma unroll
      for (int u = 0; u < 32; ++u)
        x[u] = fmaf(-s.slope, fabsf(fmaf(dir, static_cast<float>(u), d0)), y[u] * m);
    }
  } else if constexpr (kCap) {
#pragma unroll
    for (int u = 0; u < 32; u += 2)
      unpack_f32x2(mul_f32x2(pack_f32x2(y[u], y[u + 1]), mul), x[u], x[u + 1]);
  }
}

}  // namespace masked
}  // namespace vsa

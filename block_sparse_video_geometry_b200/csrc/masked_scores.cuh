// Cap and distance bias of 32 scores of a row (or column), for the forward and
// backward kernels of the dense masked attention.
#pragma once

#include "sm100.cuh"

namespace vsa {
namespace masked {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;

// Constants of a row or a call: `c` turns raw scores into log2 units, cap2 = cap
// log2(e), in = scale / cap; slope of the bias in log2 units.
struct ScoreTerms {
  float c, cap2, in, slope;
  float poly[4];               // see score_args
  float limit;                 // largest |raw score| of the polynomial
  __device__ __forceinline__ ScoreTerms(float scale, float cap, float slope_) {
    c = scale * kLog2e;
    cap2 = cap * kLog2e;
    in = cap > 0.0f ? fminf(scale / cap, 1e37f) : 0.0f;    // finite: 0 stays 0 under the smallest caps
    slope = slope_ * kLog2e;
    // c tanh(y) / y = c (1 + a1 z + a2 z^2 + a3 z^3 + a4 z^4), z = y^2 = (in x)^2, with
    // in^2 and c multiplied into the coefficients
    const float in2 = in * in;
    float f = c * in2;
    poly[0] = -0.333325982f * f;
    poly[1] = 0.133131161f * (f *= in2);
    poly[2] = -0.0522118137f * (f *= in2);
    poly[3] = 0.0156126432f * (f *= in2);
    limit = in > 0.0f && in < 1000.0f ? 0.6f / in : -1.0f;   // beyond that the coefficients could overflow
  }
};

// tanh: 1 - 2 / (1 + e^(2y)) takes two operations of the exponential unit per
// score, which then bounds the kernels, and is off by a part of 1, not of the score. For
// |y| <= 0.6 (a cap well above the scores, as caps are) tanh(y) / y is a polynomial in y^2
// on the FMA pipe: degree 4, least squares with weights driven to equal extrema, relative
// error below 2^-23; five operations a score.
// Bias: where the columns lie on one side of every row of the warp it is linear in
// the column, one operation a score. Distance of column u: |d0 + dir u|, dir = 1 or -1.
// 2 x 1,111 queries over 5,003 keys, 24 heads, cap and bias, forward: 393 us with both
// general forms in the exponential unit, 350 us so (300 us with 128-row blocks, 249 us with
// each pair's polynomial next to its exponentials, which keeps both pipes at work; 205 us
// with blocks that start and end faster).

// Largest |raw score| of 32 columns (a cap's polynomial holds up to ScoreTerms::limit).
template <bool kCap>
__device__ __forceinline__ float largest(const float (&x)[32], float top = 0.0f) {
  if constexpr (kCap) {
#pragma unroll
    for (int u = 0; u < 32; u += 2) top = fmaxf(fmaxf(top, fabsf(x[u])), fabsf(x[u + 1]));
  }
  return top;
}

// Side of `n` columns from d0: bias of column u = k (d0 + dir u); false where the
// warp's rows lie on both sides.
template <bool kBias>
__device__ __forceinline__ bool one_side(const ScoreTerms& s, float d0, float dir, float n, float& k) {
  k = 0.0f;
  if constexpr (!kBias) return true;
  const float d1 = fmaf(dir, n - 1.0f, d0);
  const bool right = __all_sync(0xffffffffu, d0 >= 0.0f && d1 >= 0.0f);
  k = right ? -s.slope : s.slope;
  return right || __all_sync(0xffffffffu, d0 <= 0.0f && d1 <= 0.0f);
}

// Log2 scores minus a reference, two columns at a time, by the polynomial and the
// linear bias.
template <bool kCap, bool kBias>
struct PairArgs {
  uint64_t c2, base, step, p0, p1, p2, p3;
  // `ref`: minus the reference where it is the same for all columns, else 0
  __device__ __forceinline__ PairArgs(const ScoreTerms& s, float k, float d0, float dir, float ref) {
    c2 = pack_f32x2(s.c, s.c);
    const float at = kBias ? fmaf(k, d0, ref) : ref;
    base = pack_f32x2(at, at);
    step = pack_f32x2(k * dir, k * dir);
    p0 = pack_f32x2(s.poly[0], s.poly[0]), p1 = pack_f32x2(s.poly[1], s.poly[1]);
    p2 = pack_f32x2(s.poly[2], s.poly[2]), p3 = pack_f32x2(s.poly[3], s.poly[3]);
  }
  // columns u and u + 1; q receives log2(e) scale tanh(y) / y
  __device__ __forceinline__ uint64_t operator()(uint64_t v, int u, uint64_t& q) const {
    q = c2;
    if constexpr (kCap) {
      const uint64_t z = mul_f32x2(v, v);
      q = fma_f32x2(fma_f32x2(fma_f32x2(fma_f32x2(p3, z, p2), z, p1), z, p0), z, c2);
    }
    uint64_t add = base;
    if constexpr (kBias) add = fma_f32x2(step, pack_f32x2(static_cast<float>(u), static_cast<float>(u + 1)), base);
    return fma_f32x2(v, q, add);
  }
};

// tanh(y) from e = 2 log2(e) y.
__device__ __forceinline__ float tanh_of(float e) { return fmaf(-2.0f, rcp_approx(1.0f + ex2_approx(e)), 1.0f); }

// Raw scores x (sums of products) -> their log2 values minus a reference (`ref`
// gives minus the reference for a pair of columns). With a cap t receives
// tanh(score / cap). What a score becomes does not depend on the scores beside it, which
// other rows see or none: where some score of the warp lies beyond the polynomial, its
// tanh comes from the general form and every other one's by the polynomial's own steps.
// (One form for the whole warp: under a cap of 10^6 a hidden score of 10^6 left the visible
// ones beside it off by 0.1. 4096 causal tokens x 24 heads with a bias, forward and backward,
// under a cap of 3: 854 us then, 1005 us now; of 50, which no score reaches, 656 and 678 us.)
template <bool kCap, bool kBias, class Ref>
__device__ __forceinline__ void score_args(float (&x)[32], float (&t)[32], const ScoreTerms& s, float d0, float dir,
                                           Ref ref) {
  float k;                      // bias of column u: k (d0 + dir u)
  const bool linear = one_side<kBias>(s, d0, dir, 32.0f, k);
  const float in_e = 2.0f * kLog2e * s.in, inv = kCap ? 1.0f / s.cap2 : 0.0f;
  const float kk = linear ? k : 0.0f;        // columns on both sides of the rows: added below
  if (!kCap || __all_sync(0xffffffffu, largest<kCap>(x) <= s.limit)) {
    const PairArgs<kCap, kBias> pair(s, kk, d0, dir, 0.0f);
#pragma unroll
    for (int u = 0; u < 32; u += 2) {
      const uint64_t v = pack_f32x2(x[u], x[u + 1]);
      uint64_t q;
      unpack_f32x2(add_f32x2(pair(v, u, q), ref(u)), x[u], x[u + 1]);
      if constexpr (kCap) unpack_f32x2(mul_f32x2(v, q), t[u], t[u + 1]);   // times 1 / cap2 below
    }
    if constexpr (kCap) {
#pragma unroll
      for (int u = 0; u < 32; ++u) t[u] *= inv;
    }
  } else if constexpr (kCap) {
#pragma unroll
    for (int u = 0; u < 32; ++u) {
      float r[2];
      unpack_f32x2(ref(u & ~1), r[0], r[1]);
      const float v = x[u], z = __fmul_rn(v, v);
      const float q = fmaf(fmaf(fmaf(fmaf(s.poly[3], z, s.poly[2]), z, s.poly[1]), z, s.poly[0]), z, s.c);
      float add = kBias ? fmaf(kk, d0, 0.0f) : 0.0f;
      if constexpr (kBias) add = fmaf(__fmul_rn(kk, dir), static_cast<float>(u), add);
      const float tanh = tanh_of(v * in_e);
      const float by_poly = __fmul_rn(__fmul_rn(v, q), inv);
      const bool near = fabsf(v) <= s.limit;
      x[u] = __fadd_rn(near ? fmaf(v, q, add) : fmaf(tanh, s.cap2, add), r[u & 1]);
      t[u] = near ? by_poly : tanh;
    }
  }
  if (kBias && !linear) {
#pragma unroll
    for (int u = 0; u < 32; ++u) x[u] = fmaf(-s.slope, fabsf(fmaf(dir, static_cast<float>(u), d0)), x[u]);
  }
}

// 2^x of a pair of columns: with `fma_pipe` on the FMA pipe, else the exponential unit.
__device__ __forceinline__ void ex2_pair(float& a, float& b, bool fma_pipe) {
  if (fma_pipe) {
    ex2_poly_f32x2(pack_f32x2(a, b), a, b);
  } else {
    a = ex2_approx(a);
    b = ex2_approx(b);
  }
}

}  // namespace masked
}  // namespace vsa

// Layer norm over the last dimension, forward and backward with the gradients
// of weight and bias.
//
// Mathematics: m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), xh = (x - m) r,
// y = xh w + b; with g = dy w: dx = r (g - mean(g) - xh mean(g xh)),
// dw = sum_rows dy xh, db = sum_rows dy. The variance is taken about the mean
// from values held in registers (a one-pass E[x^2] - m^2 loses the rows whose
// mean is far from zero).
//
// Bound: HBM (forward: x read, y written; backward: x, dy read, dx written). Every
// row is read from memory once: a short one into registers, by a group of lanes of
// one warp, the next rows' loads ahead of the current ones' arithmetic; a long one by
// one persistent block through a ring of rows in shared memory, from where the
// forward pass takes it into registers and the backward pass reads it twice (the
// sums, then dx). Backward: every thread owns fixed columns and sums dw and db of the
// rows its block passes in registers; blocks leave one partial row each, which a
// second kernel adds in a fixed order (no atomics: equal inputs give equal bits).
// Measured: 17,408 x 24 rows of 128 45 us (73% of the copy rate), backward 88 us and
// 11 us for the sums (49% together); 17,408 rows of 5,120 forward 77 us (71%),
// backward 119 us (69%) and 8 us for the sums.

#include <algorithm>
#include <cmath>

#include "sm100.cuh"
#include "vec.cuh"
#include "vsa_internal.h"

namespace vsa {
namespace {

using namespace sm100;

constexpr int kWarpBlock = 256;      // threads of a block of the short-row kernels
constexpr int kFwdBlocks = 4;        // of them per SM in the forward pass

// Rows [B, S, heads] in one index. Where the rows of every view lie at one
// stride the host gives them as [1, n, 1], which needs no division.
struct Rows {
  int64_t n;                         // B * S * heads
  int64_t S;
  int32_t heads;
  int32_t flat;
};

struct Place {
  int64_t b, s, h;
};

__device__ __forceinline__ Place place(const Rows& R, int64_t row) {
  if (R.flat) return Place{0, row, 0};
  // rows < 2^31: 32-bit divisions
  const uint32_t r = static_cast<uint32_t>(row), t = r / static_cast<uint32_t>(R.heads);
  Place p;
  p.h = r - t * static_cast<uint32_t>(R.heads);
  p.b = t / static_cast<uint32_t>(R.S);
  p.s = t - static_cast<uint32_t>(p.b) * static_cast<uint32_t>(R.S);
  return p;
}

__device__ __forceinline__ int64_t offset(const Strides& st, const Place& p) {
  return p.b * st.b + p.s * st.s + p.h * st.h;
}

struct FwdArgs {
  Rows R;
  const void* x;
  void* y;
  const void *w, *b;
  float *mean, *rstd;
  Strides sx, sy;
  int width, w_f32, w_wide;
  float eps, inv_n;
};

struct BwdArgs {
  Rows R;
  const void *dy, *x, *w;
  const float *mean, *rstd;
  void* dx;
  Strides sdy, sx, sdx;
  float* part;                       // [blocks][2][width] partial dw, db, or null
  int width, w_f32, w_wide, dx_f32;
  float inv_n;
};

// Weight or bias values of VEC columns from c, stored as float or T; with
// `w_wide` in one access (16-byte aligned vectors).
template <class T, int VEC>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, int w_wide, int c, float (&v)[VEC]) {
  if (w_f32 || sizeof(T) == 4) {
    const float* p = static_cast<const float*>(w) + c;
    if (w_wide) {
      Pack<float, VEC> k;
      k.load(p);
      k.get(v);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = __ldg(p + i);
    }
  } else {
    const T* p = static_cast<const T*>(w) + c;
    if (w_wide) {
      Pack<T, VEC> k;
      k.load(p);
      k.get(v);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = to_f32(p[i]);
    }
  }
}

// Weight and bias of vector c (1 and 0 where there are none).
template <class T, int VEC>
__device__ __forceinline__ void weights(const FwdArgs& a, int c, int nv, float (&w)[VEC], float (&b)[VEC]) {
#pragma unroll
  for (int j = 0; j < VEC; ++j) w[j] = 1.0f, b[j] = 0.0f;
  if (a.w && c < nv) load_weight<T, VEC>(a.w, a.w_f32, a.w_wide, c * VEC, w);
  if (a.b && c < nv) load_weight<T, VEC>(a.b, a.w_f32, a.w_wide, c * VEC, b);
}

template <int LANES>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum over the block, in every thread. `buf` holds one float per warp and is
// not rewritten before the block's next barrier.
__device__ __forceinline__ float block_sum(float x, float* buf) {
  x = lane_sum<32>(x);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return x;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return lane_sum<32>(lane < warps ? buf[lane] : 0.0f);
}

template <int N>
__device__ __forceinline__ float sum_of(const float (&x)[N]) {
  uint64_t s2 = 0;
  float s = 0.0f, t = 0.0f;
  each<N>([&](int i) { s2 = add_f32x2(s2, pack_f32x2(x[i], x[i + 1])); }, [&](int i) { s += x[i]; });
  if constexpr (N % 2 == 0) unpack_f32x2(s2, s, t);
  return s + t;
}

// The single-element forms round every step (no fused operations): a row of one or
// two elements has a gradient that cancels to nothing, and so it does here, as the
// formula does step by step.

// x = x - m in place; returns the sum of squares.
template <int N>
__device__ __forceinline__ float centre(float (&x)[N], float m) {
  uint64_t s2 = 0;
  float s = 0.0f, t = 0.0f;
  const uint64_t m2 = pack_f32x2(-m, -m);
  each<N>(
      [&](int i) {
        const uint64_t d = add_f32x2(pack_f32x2(x[i], x[i + 1]), m2);
        s2 = fma_f32x2(d, d, s2);
        unpack_f32x2(d, x[i], x[i + 1]);
      },
      [&](int i) {
        x[i] = __fsub_rn(x[i], m);
        s = __fadd_rn(s, __fmul_rn(x[i], x[i]));
      });
  if constexpr (N % 2 == 0) unpack_f32x2(s2, s, t);
  return s + t;
}

// x = x * (r w) + b in place.
template <int N>
__device__ __forceinline__ void scale_shift(float (&x)[N], float r, const float (&w)[N], const float (&b)[N]) {
  const uint64_t r2 = pack_f32x2(r, r);
  each<N>(
      [&](int i) {
        const uint64_t a = mul_f32x2(r2, pack_f32x2(w[i], w[i + 1]));
        unpack_f32x2(fma_f32x2(pack_f32x2(x[i], x[i + 1]), a, pack_f32x2(b[i], b[i + 1])), x[i], x[i + 1]);
      },
      [&](int i) { x[i] = fmaf(x[i], r * w[i], b[i]); });
}

// ------------------------------------------------------------------ forward
// Short rows: LANES lanes of a warp per row, E vectors of VEC elements each (vector
// i of lane t is i * LANES + t). Persistent blocks keep the weights in registers and
// fetch the next U rows of a lane group while they work on the current ones.
template <class T, int VEC, int E, int LANES, int U>
__global__ void __launch_bounds__(kWarpBlock, E == 1 ? kFwdBlocks : 2)
norm_fwd_warp_kernel(const __grid_constant__ FwdArgs a) {
  constexpr int kGroups = kWarpBlock / LANES;
  const int t = threadIdx.x % LANES, group = threadIdx.x / LANES, nv = a.width / VEC;
  float w[E][VEC], b[E][VEC];
#pragma unroll
  for (int i = 0; i < E; ++i) weights<T, VEC>(a, i * LANES + t, nv, w[i], b[i]);
  Pack<T, VEC> next[U][E];
  auto fetch = [&](int64_t r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r0 + u * kGroups + group;
      if (row >= a.R.n) continue;
      const T* x = static_cast<const T*>(a.x) + offset(a.sx, place(a.R, row));
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i * LANES + t < nv) next[u][i].load(x + (i * LANES + t) * VEC);
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups * U;
  int64_t r0 = static_cast<int64_t>(blockIdx.x) * kGroups * U;
  fetch(r0);
  for (; r0 < a.R.n; r0 += step) {
    Pack<T, VEC> k[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < E; ++i) k[u][i] = next[u][i];
    fetch(r0 + step);                                // y may lie over x: other rows
    float v[U][E][VEC], mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mean[u] = 0.0f;
      if (r0 + u * kGroups + group >= a.R.n) continue;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (i * LANES + t >= nv) continue;
        k[u][i].get(v[u][i]);
        mean[u] += sum_of(v[u][i]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) mean[u] = lane_sum<LANES>(mean[u]) * a.inv_n;     // every lane takes part
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rstd[u] = 0.0f;
      if (r0 + u * kGroups + group >= a.R.n) continue;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i * LANES + t < nv) rstd[u] += centre(v[u][i], mean[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) rstd[u] = rsqrtf(lane_sum<LANES>(rstd[u]) * a.inv_n + a.eps);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r0 + u * kGroups + group;
      if (row >= a.R.n) continue;
      T* y = static_cast<T*>(a.y) + offset(a.sy, place(a.R, row));
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (i * LANES + t >= nv) continue;
        scale_shift(v[u][i], rstd[u], w[i], b[i]);
        k[u][i].set(v[u][i]);
        k[u][i].store(y + (i * LANES + t) * VEC);
      }
      if (t == 0 && a.mean) {
        a.mean[row] = mean[u];
        a.rstd[row] = rstd[u];
      }
    }
  }
}

// Asynchronous copy of one vector into this thread's own place in shared memory
// (of 4 or 16 bytes; 2-byte elements one by one are copied at once).
template <int BYTES>
__device__ __forceinline__ void stage_in(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  } else if constexpr (BYTES == 32) {
    stage_in<16>(dst, src);
    stage_in<16>(static_cast<char*>(dst) + 16, static_cast<const char*>(src) + 16);
  } else if constexpr (BYTES == 4) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
  } else {
    static_assert(BYTES == 2);
    *static_cast<uint16_t*>(dst) = *static_cast<const uint16_t*>(src);
  }
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 2-byte rows that start anywhere (odd widths, shifted views) are staged in the
// aligned 16-byte pieces that they cover, the elements before the first and behind
// the last whole piece one by one, so that nothing outside the row is read. Element
// c of a row at address p comes to lie (p % 16) / size + c elements into the stage.
// (One element per copy instead: 1000 us for 7,825 bf16 rows of 9,009.)
__host__ __device__ constexpr int loose_pitch(int width, int size) { return (width * size + 15) / 16 * 16 + 16; }
template <class T>
__device__ __forceinline__ int loose_shift(const T* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T));
}
template <class T>
__device__ __forceinline__ void stage_loose(uint8_t* stage, const T* p, int width) {
  const int shift = loose_shift(p), pieces = (shift + width + 16 / static_cast<int>(sizeof(T)) - 1) * static_cast<int>(sizeof(T)) / 16;
  const T* base = p - shift;
  constexpr int kN = 16 / static_cast<int>(sizeof(T));
  for (int k = threadIdx.x; k < pieces; k += blockDim.x) {
    const int c0 = k * kN - shift;
    if (c0 >= 0 && c0 + kN <= width) {
      stage_in<16>(stage + 16 * k, base + k * kN);
    } else {
      for (int j = max(c0, 0); j < min(c0 + kN, width); ++j) reinterpret_cast<T*>(stage)[shift + j] = p[j];
    }
  }
}

// Long rows: one block per row, E vectors of VEC elements per thread (vector i of
// thread t is i * threads + t). A persistent block keeps up to three rows ahead on
// their way into shared memory; a thread reads back only what it copied itself,
// so the ring needs no barrier (loose rows need one). Rows of the ring: four where `bytes` a thread and
// row times `threads` allow it.
__host__ __device__ constexpr int ring_rows(int bytes, int threads) {
  const int n = (200 << 10) / (bytes * threads);
  return n < 1 ? 1 : n > 4 ? 4 : n;
}
template <class T, int VEC, int E, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const __grid_constant__ FwdArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kRing = ring_rows(sizeof(T) * VEC * E, MAXT);
  constexpr bool kLoose = VEC == 1 && sizeof(T) == 2;
  __shared__ float red[2][2][32];
  using P = Pack<T, VEC>;
  P* mine = reinterpret_cast<P*>(ring) + threadIdx.x;
  const int tpr = blockDim.x, t = threadIdx.x, nv = a.width / VEC;
  const int pitch = loose_pitch(a.width, sizeof(T));
  auto fetch = [&](int64_t row, int st) {
    if (row < a.R.n) {
      const T* x = static_cast<const T*>(a.x) + offset(a.sx, place(a.R, row));
      if constexpr (kLoose) {
        stage_loose(ring + st * pitch, x, a.width);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (i * tpr + t < nv) stage_in<sizeof(P)>(mine + (st * E + i) * tpr, x + static_cast<int64_t>(i * tpr + t) * VEC);
      }
    }
    stage_commit();
  };
  float w[E][VEC], b[E][VEC];
#pragma unroll
  for (int i = 0; i < E; ++i) weights<T, VEC>(a, i * tpr + t, nv, w[i], b[i]);
  int st = 0, phase = 0;
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(blockIdx.x + static_cast<int64_t>(i) * gridDim.x, i);
  for (int64_t row = blockIdx.x; row < a.R.n; row += gridDim.x) {
    if constexpr (kRing == 1) {
      if constexpr (kLoose) __syncthreads();               // the row before was read by all threads
      fetch(row, 0);
    }
    stage_wait<(kRing > 2 ? kRing - 2 : 0)>();
    const T* loose = nullptr;
    if constexpr (kLoose) {
      __syncthreads();                                       // pieces of all threads
      loose = reinterpret_cast<const T*>(ring + st * pitch) +
              loose_shift(static_cast<const T*>(a.x) + offset(a.sx, place(a.R, row)));
    }
    float v[E][VEC], sum = 0.0f, sq = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (i * tpr + t >= nv) continue;
      if constexpr (kLoose) v[i][0] = to_f32(loose[i * tpr + t]);
      else mine[(st * E + i) * tpr].get(v[i]);
      sum += sum_of(v[i]);
    }
    if constexpr (kRing > 1) fetch(row + static_cast<int64_t>(kRing - 1) * gridDim.x, st == 0 ? kRing - 1 : st - 1);
    if (++st == kRing) st = 0;
    const float mean = block_sum(sum, red[phase][0]) * a.inv_n;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (i * tpr + t < nv) sq += centre(v[i], mean);
    }
    const float rstd = rsqrtf(block_sum(sq, red[phase][1]) * a.inv_n + a.eps);
    phase ^= 1;
    T* y = static_cast<T*>(a.y) + offset(a.sy, place(a.R, row));
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = i * tpr + t;
      if (c >= nv) continue;
      scale_shift(v[i], rstd, w[i], b[i]);
      P k;
      k.set(v[i]);
      k.store(y + static_cast<int64_t>(c) * VEC);
    }
    if (t == 0 && a.mean) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
  }
  stage_wait<0>();
}

// ----------------------------------------------------------------- backward
// A thread's vector of columns: the sums dw and db of the rows it passed. The row
// itself is unpacked again for the second pass: unpacked it would not fit.
template <class T, class G, int VEC>
struct Columns {
  float w[VEC], dw[VEC], db[VEC];
  __device__ __forceinline__ void start(const BwdArgs& a, int c, int nv) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = 1.0f, dw[j] = db[j] = 0.0f;
    if (a.w && c < nv) load_weight<T, VEC>(a.w, a.w_f32, a.w_wide, c * VEC, w);
  }
  // adds a row's share of dw and db, and of the two sums over the row
  __device__ __forceinline__ void add(const Pack<T, VEC>& kx, const Pack<G, VEC>& kg,
                                      float mean, float rstd, float& s1, float& s2) {
    float x[VEC], g[VEC];
    kx.get(x);
    kg.get(g);
    const uint64_t m2 = pack_f32x2(-mean, -mean), r2 = pack_f32x2(rstd, rstd);
    uint64_t a1 = 0, a2 = 0;
    float b1 = 0.0f, b2 = 0.0f, t1 = 0.0f, t2 = 0.0f;
    each<VEC>(
        [&](int i) {
          const uint64_t xh = mul_f32x2(add_f32x2(pack_f32x2(x[i], x[i + 1]), m2), r2);
          const uint64_t d = pack_f32x2(g[i], g[i + 1]), y = mul_f32x2(d, pack_f32x2(w[i], w[i + 1]));
          unpack_f32x2(fma_f32x2(d, xh, pack_f32x2(dw[i], dw[i + 1])), dw[i], dw[i + 1]);
          unpack_f32x2(add_f32x2(d, pack_f32x2(db[i], db[i + 1])), db[i], db[i + 1]);
          a1 = add_f32x2(a1, y);
          a2 = fma_f32x2(y, xh, a2);
        },
        [&](int i) {
          const float xh = __fmul_rn(__fsub_rn(x[i], mean), rstd), y = __fmul_rn(g[i], w[i]);
          dw[i] = fmaf(g[i], xh, dw[i]);
          db[i] += g[i];
          b1 = __fadd_rn(b1, y);
          b2 = __fadd_rn(b2, __fmul_rn(y, xh));
        });
    if constexpr (VEC % 2 == 0) {
      unpack_f32x2(a1, b1, t1);
      unpack_f32x2(a2, b2, t2);
    }
    s1 += b1 + t1;
    s2 += b2 + t2;
  }
  // rstd (g - c1 - xh c2)
  __device__ __forceinline__ void write(const BwdArgs& a, const Pack<T, VEC>& kx, const Pack<G, VEC>& kg,
                                               float mean, float rstd, float c1, float c2, int64_t at) {
    float x[VEC], g[VEC];
    kx.get(x);
    kg.get(g);
    const uint64_t m2 = pack_f32x2(-mean, -mean), r2 = pack_f32x2(rstd, rstd);
    const uint64_t n1 = pack_f32x2(-c1, -c1), n2 = pack_f32x2(-c2, -c2);
    each<VEC>(
        [&](int i) {
          const uint64_t xh = mul_f32x2(add_f32x2(pack_f32x2(x[i], x[i + 1]), m2), r2);
          const uint64_t y = fma_f32x2(pack_f32x2(g[i], g[i + 1]), pack_f32x2(w[i], w[i + 1]), fma_f32x2(xh, n2, n1));
          unpack_f32x2(mul_f32x2(r2, y), g[i], g[i + 1]);
        },
        [&](int i) {
          const float xh = __fmul_rn(__fsub_rn(x[i], mean), rstd);
          g[i] = __fmul_rn(rstd, __fsub_rn(__fsub_rn(__fmul_rn(g[i], w[i]), c1), __fmul_rn(xh, c2)));
        });
    if (a.dx_f32) {
      Pack<float, VEC> k;
      k.set(g);
      k.store(static_cast<float*>(a.dx) + at);
    } else {
      Pack<T, VEC> k;
      k.set(g);
      k.store(static_cast<T*>(a.dx) + at);
    }
  }
};

// Short rows, as in the forward kernel; the next row is fetched into registers
// while the current one is worked on.
template <class T, class G, int VEC, int E, int LANES>
__global__ void __launch_bounds__(kWarpBlock) norm_bwd_warp_kernel(const __grid_constant__ BwdArgs a) {
  constexpr int kGroups = kWarpBlock / LANES;
  const int t = threadIdx.x % LANES, group = threadIdx.x / LANES, nv = a.width / VEC;
  Columns<T, G, VEC> col[E];
#pragma unroll
  for (int i = 0; i < E; ++i) col[i].start(a, i * LANES + t, nv);
  Pack<T, VEC> kx[E];
  Pack<G, VEC> kg[E];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t row) {
    if (row >= a.R.n) return;
    const Place p = place(a.R, row);
    const T* x = static_cast<const T*>(a.x) + offset(a.sx, p);
    const G* dy = static_cast<const G*>(a.dy) + offset(a.sdy, p);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (i * LANES + t >= nv) continue;
      kx[i].load(x + (i * LANES + t) * VEC);
      kg[i].load(dy + (i * LANES + t) * VEC);
    }
    mean = a.mean[row];
    rstd = a.rstd[row];
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t r0 = static_cast<int64_t>(blockIdx.x) * kGroups;
  fetch(r0 + group);
  for (; r0 < a.R.n; r0 += step) {
    const int64_t row = r0 + group;
    const bool live = row < a.R.n;                   // every lane takes part in the sums
    const float m = mean, r = rstd;
    float s1 = 0.0f, s2 = 0.0f;
    Pack<T, VEC> cx[E];
    Pack<G, VEC> cg[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      cx[i] = kx[i];
      cg[i] = kg[i];
      if (live && i * LANES + t < nv) col[i].add(cx[i], cg[i], m, r, s1, s2);
    }
    // dx may lie over dy: a row is fetched and written by the same lanes, in that order
    fetch(row + step);
    s1 = lane_sum<LANES>(s1) * a.inv_n;
    s2 = lane_sum<LANES>(s2) * a.inv_n;
    if (!live) continue;
    const int64_t od = offset(a.sdx, place(a.R, row));
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i * LANES + t < nv) col[i].write(a, cx[i], cg[i], m, r, s1, s2, od + (i * LANES + t) * VEC);
  }
  if (!a.part) return;
  // the block's row groups first, in group order
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
  __shared__ float acc[2][LANES * E * VEC];
  for (int i = threadIdx.x; i < 2 * LANES * E * VEC; i += kWarpBlock) (&acc[0][0])[i] = 0.0f;
  for (int gidx = 0; gidx < kGroups; ++gidx) {
    __syncthreads();
    if (group != gidx) continue;
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        acc[0][(i * LANES + t) * VEC + j] += col[i].dw[j];
        acc[1][(i * LANES + t) * VEC + j] += col[i].db[j];
      }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.width; c += kWarpBlock) {
    part[c] = acc[0][c];
    part[a.width + c] = acc[1][c];
  }
}

// Long rows: one persistent block per row, its next rows on their way into shared
// memory as in the forward kernel.
template <class T, class G, int VEC, int E, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const __grid_constant__ BwdArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr int kRing = ring_rows((sizeof(T) + sizeof(G)) * VEC * E, MAXT);
  constexpr bool kLoose = VEC == 1 && sizeof(T) == 2;
  __shared__ float red[2][2][32];
  using PX = Pack<T, VEC>;
  using PG = Pack<G, VEC>;
  const int tpr = blockDim.x, t = threadIdx.x, nv = a.width / VEC;
  PX* my_x = reinterpret_cast<PX*>(ring) + t;
  PG* my_g = reinterpret_cast<PG*>(ring + sizeof(PX) * kRing * E * tpr) + t;
  const int pitch_x = loose_pitch(a.width, sizeof(T)), pitch = pitch_x + loose_pitch(a.width, sizeof(G));
  auto fetch = [&](int64_t row, int st) {
    if (row < a.R.n) {
      const Place p = place(a.R, row);
      const T* x = static_cast<const T*>(a.x) + offset(a.sx, p);
      const G* dy = static_cast<const G*>(a.dy) + offset(a.sdy, p);
      if constexpr (kLoose) {
        stage_loose(ring + st * pitch, x, a.width);
        stage_loose(ring + st * pitch + pitch_x, dy, a.width);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int64_t c = i * tpr + t;
          if (c >= nv) continue;
          stage_in<sizeof(PX)>(my_x + (st * E + i) * tpr, x + c * VEC);
          stage_in<sizeof(PG)>(my_g + (st * E + i) * tpr, dy + c * VEC);
        }
      }
    }
    stage_commit();
  };
  Columns<T, G, VEC> col[E];
#pragma unroll
  for (int i = 0; i < E; ++i) col[i].start(a, i * tpr + t, nv);
  int st = 0, phase = 0;
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(blockIdx.x + static_cast<int64_t>(i) * gridDim.x, i);
  float mean = 0.0f, rstd = 0.0f;
  if (blockIdx.x < a.R.n) {
    mean = a.mean[blockIdx.x];
    rstd = a.rstd[blockIdx.x];
  }
  for (int64_t row = blockIdx.x; row < a.R.n; row += gridDim.x) {
    const int64_t next = row + gridDim.x;
    const float next_mean = next < a.R.n ? a.mean[next] : 0.0f, next_rstd = next < a.R.n ? a.rstd[next] : 0.0f;
    if constexpr (kRing == 1) {
      if constexpr (kLoose) __syncthreads();               // the row before was read by all threads
      fetch(row, 0);
    }
    stage_wait<(kRing > 2 ? kRing - 2 : 0)>();
    const T* lx = nullptr;
    const G* lg = nullptr;
    if constexpr (kLoose) {
      __syncthreads();                                       // pieces of all threads
      const Place p = place(a.R, row);
      lx = reinterpret_cast<const T*>(ring + st * pitch) + loose_shift(static_cast<const T*>(a.x) + offset(a.sx, p));
      lg = reinterpret_cast<const G*>(ring + st * pitch + pitch_x) +
           loose_shift(static_cast<const G*>(a.dy) + offset(a.sdy, p));
    }
    auto vec_x = [&](int i) {
      if constexpr (kLoose) {
        PX k;
        k.t[0] = lx[i * tpr + t];
        return k;
      } else {
        return my_x[(st * E + i) * tpr];
      }
    };
    auto vec_g = [&](int i) {
      if constexpr (kLoose) {
        PG k;
        k.t[0] = lg[i * tpr + t];
        return k;
      } else {
        return my_g[(st * E + i) * tpr];
      }
    };
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i * tpr + t < nv)
        col[i].add(vec_x(i), vec_g(i), mean, rstd, s1, s2);
    // dx may lie over dy: a row is fetched and written by the same block, in that order
    if constexpr (kRing > 1) fetch(row + static_cast<int64_t>(kRing - 1) * gridDim.x, st == 0 ? kRing - 1 : st - 1);
    s1 = lane_sum<32>(s1);
    s2 = lane_sum<32>(s2);
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (warps > 1) {
      if (lane == 0) {
        red[phase][0][threadIdx.x >> 5] = s1;
        red[phase][1][threadIdx.x >> 5] = s2;
      }
      __syncthreads();
      s1 = lane_sum<32>(lane < warps ? red[phase][0][lane] : 0.0f);
      s2 = lane_sum<32>(lane < warps ? red[phase][1][lane] : 0.0f);
      phase ^= 1;
    }
    s1 *= a.inv_n;
    s2 *= a.inv_n;
    const int64_t od = offset(a.sdx, place(a.R, row));
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int64_t c = i * tpr + t;
      if (c < nv)
        col[i].write(a, vec_x(i), vec_g(i), mean, rstd, s1, s2,
                     od + c * VEC);
    }
    if (++st == kRing) st = 0;
    mean = next_mean;
    rstd = next_rstd;
  }
  stage_wait<0>();
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = i * tpr + t;
    if (c >= nv) continue;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      part[c * VEC + j] = col[i].dw[j];
      part[a.width + c * VEC + j] = col[i].db[j];
    }
  }
}

// dweight and dbias from the blocks' partial rows: 32 columns per block, 32 rows
// of threads each adding every 32nd partial, then a tree over the 32.
constexpr int kSumCols = 32, kSumRows = 32;
__global__ void __launch_bounds__(kSumCols * kSumRows)
norm_sum_kernel(const float* __restrict__ part, int n_part, int width, float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float acc[kSumRows][kSumCols + 1];
  const int cc = threadIdx.x % kSumCols, c = blockIdx.x * kSumCols + cc, r = threadIdx.x / kSumCols;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;                                 // the whole block
  float s = 0.0f;
  if (c < width) {
    const float* p = part + static_cast<int64_t>(blockIdx.y) * width + c;
#pragma unroll 8
    for (int i = r; i < n_part; i += kSumRows) s += p[static_cast<int64_t>(i) * 2 * width];
  }
  acc[r][cc] = s;
  __syncthreads();
  const float x = lane_sum<32>(acc[cc][r]);         // row r now sums column r
  const int col = blockIdx.x * kSumCols + r;
  if (cc == 0 && col < width) out[col] = x;
}

// ------------------------------------------------------------------ launches
// Few vectors of the widest aligned access: lanes of one warp per row. Else one
// block per row with `ept` elements per thread: 16 from a width of 2048 on where
// rows fill the GPU (17,408 x 5120 forward and backward: 209 us; 8: 318 us, the
// row's fixed work of sums and addresses; 32: 250 us, too few threads beside their
// registers), 8 for narrower or few rows, 32 above 8192.
struct Shape {
  int vec, lanes;         // lanes 64: one block per row
  int ept;
  int threads, rows_per_block;
};
constexpr int kFwdU = 2;   // rows in flight per lane group of the short-row forward kernel

Shape shape_of(int width, int vec, int64_t rows, int u) {
  const int nv = width / vec;
  if (nv <= 32 || (vec == 1 && width <= 512)) {
    // vectors per lane: 1, or for single elements up to 16
    const int lanes = nv <= 16 ? 16 : 32, e = nv <= 32 ? 1 : nv <= 128 ? 4 : 16;
    return Shape{vec, lanes, e * vec, kWarpBlock, kWarpBlock / lanes * (e == 1 ? u : 1)};
  }
  const int ept = width > 8192 ? 32 : width >= 2048 && rows >= 512 ? 16 : 8, e = ept / vec;
  return Shape{vec, 64, ept, ((nv + e - 1) / e + 31) / 32 * 32, 1};
}

constexpr int kMaxSms = 160;                        // the workspace is sized for this many
// Persistent blocks: as many per SM as make about `threads` threads, at most 8.
int persistent(int64_t rows, const Shape& s, int threads, int sms) {
  const int per_sm = std::max(1, std::min(8, threads / s.threads));
  const int64_t most = static_cast<int64_t>(std::min(sms, kMaxSms)) * per_sm;
  return static_cast<int>(std::min<int64_t>((rows + s.rows_per_block - 1) / s.rows_per_block, most));
}

template <class K, class A>
vsa_status start(const char* where, K kernel, int blocks, int threads, size_t smem, const A& a, cudaStream_t stream) {
  if (smem > (40u << 10)) {                          // with a block's static shared memory above 48 KB
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_fail(where, e);
  }
  kernel<<<blocks, threads, smem, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK : cuda_fail(where, e);
}

template <class T, int VEC>
vsa_status fwd_launch(const Shape& s, const FwdArgs& a, cudaStream_t stream) {
  const char* where = "vsa_layer_norm_fwd";
  const bool wide = s.ept == VEC;                          // of the warp kernels: one vector per lane
  const int n = persistent(a.R.n, s, s.lanes > 32 ? 960 : (wide ? kFwdBlocks : 2) * kWarpBlock, device_sms());
  if (s.lanes == 16) return start(where, norm_fwd_warp_kernel<T, VEC, 1, 16, kFwdU>, n, s.threads, 0, a, stream);
  if (s.lanes == 32 && wide) return start(where, norm_fwd_warp_kernel<T, VEC, 1, 32, kFwdU>, n, s.threads, 0, a, stream);
  if constexpr (VEC == 1) {
    if (s.lanes == 32 && s.ept == 4) return start(where, norm_fwd_warp_kernel<T, 1, 4, 32, 1>, n, s.threads, 0, a, stream);
    if (s.lanes == 32) return start(where, norm_fwd_warp_kernel<T, 1, 16, 32, 1>, n, s.threads, 0, a, stream);
  }
  const int row = static_cast<int>(sizeof(T)) * s.ept;
  auto smem = [&](int most) { return (static_cast<size_t>(row) * s.threads + 32) * ring_rows(row, most); };
  if (s.ept == 8) return start(where, norm_fwd_kernel<T, VEC, 8 / VEC, 1024>, n, s.threads, smem(1024), a, stream);
  if (s.ept == 16) return start(where, norm_fwd_kernel<T, VEC, 16 / VEC, 512>, n, s.threads, smem(512), a, stream);
  return start(where, norm_fwd_kernel<T, VEC, 32 / VEC, 512>, n, s.threads, smem(512), a, stream);
}

// Blocks of the backward kernel: a partial row each.
int bwd_blocks(int64_t rows, const Shape& s, int sms) {
  return persistent(rows, s, s.lanes > 32 ? 640 : (s.ept > 8 ? 2 : 4) * kWarpBlock, sms);
}

template <class T, class G, int VEC>
vsa_status bwd_launch(const Shape& s, const BwdArgs& a, int blocks, cudaStream_t stream) {
  const char* where = "vsa_layer_norm_bwd";
  if (s.lanes == 16) return start(where, norm_bwd_warp_kernel<T, G, VEC, 1, 16>, blocks, s.threads, 0, a, stream);
  if (s.lanes == 32 && s.ept == VEC)
    return start(where, norm_bwd_warp_kernel<T, G, VEC, 1, 32>, blocks, s.threads, 0, a, stream);
  if constexpr (VEC == 1) {
    if (s.lanes == 32 && s.ept == 4)
      return start(where, norm_bwd_warp_kernel<T, G, 1, 4, 32>, blocks, s.threads, 0, a, stream);
    if (s.lanes == 32) return start(where, norm_bwd_warp_kernel<T, G, 1, 16, 32>, blocks, s.threads, 0, a, stream);
  }
  const int row = static_cast<int>(sizeof(T) + sizeof(G)) * s.ept;
  auto smem = [&](int most) { return (static_cast<size_t>(row) * s.threads + 64) * ring_rows(row, most); };
  if (s.ept == 8)
    return start(where, norm_bwd_kernel<T, G, VEC, 8 / VEC, 1024>, blocks, s.threads, smem(1024), a, stream);
  if (s.ept == 16)
    return start(where, norm_bwd_kernel<T, G, VEC, 16 / VEC, 512>, blocks, s.threads, smem(512), a, stream);
  return start(where, norm_bwd_kernel<T, G, VEC, 32 / VEC, 512>, blocks, s.threads, smem(512), a, stream);
}

// Rows at one stride in all views: [1, n, 1].
bool flat_rows(const Strides& st, int32_t B, int64_t S, int32_t heads, int64_t* stride) {
  *stride = heads > 1 ? st.h : S > 1 ? st.s : st.b;
  if (heads > 1 && S > 1 && st.s != heads * st.h) return false;
  return B == 1 || (heads == 1 && S == 1) || st.b == *stride * heads * S;
}

template <class... V>
void flatten(Rows* R, int32_t B, int64_t S, V*... views) {
  int64_t stride[sizeof...(V)];
  int i = 0;
  if (!(flat_rows(*views, B, S, R->heads, &stride[i++]) && ...)) return;
  i = 0;
  ((*views = Strides{0, stride[i++], 0}), ...);
  R->flat = 1;
}

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Elements per access that every row of the views allows: 16 bytes of `elem`
// byte elements when all rows start on a multiple of that many elements and the
// width is one, else single elements.
bool vec_ok(const vsa_view* v, const Strides& st, int vec, int32_t width) {
  return width % vec == 0 && st.b % vec == 0 && st.s % vec == 0 && st.h % vec == 0 &&
         aligned(v->data, std::min<int64_t>(16, vec * static_cast<int64_t>(dtype_bytes(v->dtype))));
}

vsa_status check_rows(int32_t B, int64_t S, int32_t heads, int32_t width, Rows* R) {
  if (B < 0 || S < 0 || heads <= 0 || width <= 0) return VSA_ERR_INVALID_ARG;
  if (width > VSA_MAX_NORM_WIDTH) return VSA_ERR_UNSUPPORTED;
  if (B > 0 && S > INT32_MAX / B) return VSA_ERR_UNSUPPORTED;
  if (S * B > INT32_MAX / heads) return VSA_ERR_UNSUPPORTED;
  R->n = static_cast<int64_t>(B) * S * heads;
  R->S = S;
  R->heads = heads;
  R->flat = 0;
  return VSA_OK;
}

}  // namespace
}  // namespace vsa

using namespace vsa;

extern "C" {

vsa_status vsa_layer_norm_fwd(int32_t B, int64_t S, int32_t width, const vsa_view* x, const void* weight,
                              const void* bias, int32_t weight_dtype, float eps, const vsa_view* y, float* mean,
                              float* rstd, cudaStream_t stream) {
  if (!x || !y) return VSA_ERR_INVALID_ARG;
  FwdArgs a{};
  vsa_status st = check_rows(B, S, x->heads, width, &a.R);
  if (st == VSA_OK) st = check_view(x, B, S, width, 1, false);
  if (st == VSA_OK) st = check_view(y, B, S, width, 1, true);
  if (st != VSA_OK) return st;
  if (y->heads != x->heads || y->dtype != x->dtype) return VSA_ERR_INVALID_ARG;
  if ((weight || bias) && weight_dtype != x->dtype && weight_dtype != VSA_F32) return VSA_ERR_INVALID_ARG;
  const int64_t wsize = static_cast<int64_t>(dtype_bytes(weight_dtype));
  if ((weight && !aligned(weight, wsize)) || (bias && !aligned(bias, wsize))) return VSA_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return VSA_ERR_INVALID_ARG;
  if ((mean == nullptr) != (rstd == nullptr) || !aligned(mean, 4) || !aligned(rstd, 4)) return VSA_ERR_INVALID_ARG;
  if (a.R.n == 0) return VSA_OK;
  a.x = x->data;
  a.y = y->data;
  a.w = weight;
  a.b = bias;
  a.w_f32 = weight_dtype == VSA_F32;
  a.w_wide = aligned(weight, 16) && aligned(bias, 16);
  a.mean = mean;
  a.rstd = rstd;
  a.sx = view_strides(x, B, S);
  a.sy = view_strides(y, B, S);
  flatten(&a.R, B, S, &a.sx, &a.sy);
  a.width = width;
  a.eps = eps;
  a.inv_n = 1.0f / static_cast<float>(width);
  const int vec = 16 / static_cast<int>(dtype_bytes(x->dtype));
  const bool wide = vec_ok(x, a.sx, vec, width) && vec_ok(y, a.sy, vec, width);
  const Shape s = shape_of(width, wide ? vec : 1, a.R.n, kFwdU);
  if (x->dtype == VSA_F32) return wide ? fwd_launch<float, 4>(s, a, stream) : fwd_launch<float, 1>(s, a, stream);
  if (x->dtype == VSA_BF16) return wide ? fwd_launch<bf16, 8>(s, a, stream) : fwd_launch<bf16, 1>(s, a, stream);
  return wide ? fwd_launch<f16, 8>(s, a, stream) : fwd_launch<f16, 1>(s, a, stream);
}

vsa_status vsa_layer_norm_bwd_workspace_size(int32_t B, int64_t S, int32_t heads, int32_t width, size_t* bytes) {
  Rows R;
  if (!bytes) return VSA_ERR_INVALID_ARG;
  const vsa_status st = check_rows(B, S, heads, width, &R);
  if (st != VSA_OK) return st;
  // a partial row of dw and db per block, of the access (single elements, 4 or 8) with the
  // most blocks: types and alignment are not at hand
  int blocks = 1;
  for (int vec : {1, 4, 8})
    if (width % vec == 0) blocks = std::max(blocks, bwd_blocks(R.n, shape_of(width, vec, R.n, 1), kMaxSms));
  *bytes = align_up(static_cast<size_t>(blocks) * 2 * width * sizeof(float), 256);
  return VSA_OK;
}

vsa_status vsa_layer_norm_bwd(int32_t B, int64_t S, int32_t width, const vsa_view* dy, const vsa_view* x,
                              const void* weight, int32_t weight_dtype, const float* mean, const float* rstd,
                              const vsa_view* dx, float* dweight, float* dbias, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  if (!x || !dy || !dx) return VSA_ERR_INVALID_ARG;
  BwdArgs a{};
  vsa_status st = check_rows(B, S, x->heads, width, &a.R);
  if (st == VSA_OK) st = check_view(x, B, S, width, 1, false);
  if (st == VSA_OK) st = check_view(dy, B, S, width, 1, false);
  if (st == VSA_OK) st = check_view(dx, B, S, width, 1, true);
  if (st != VSA_OK) return st;
  if (dy->heads != x->heads || dx->heads != x->heads) return VSA_ERR_INVALID_ARG;
  for (const vsa_view* v : {dy, dx})
    if (v->dtype != x->dtype && v->dtype != VSA_F32) return VSA_ERR_INVALID_ARG;
  if (weight && weight_dtype != x->dtype && weight_dtype != VSA_F32) return VSA_ERR_INVALID_ARG;
  if (weight && !aligned(weight, static_cast<int64_t>(dtype_bytes(weight_dtype)))) return VSA_ERR_INVALID_ARG;
  if (!aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4)) return VSA_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256) return VSA_ERR_INVALID_ARG;
  size_t need = 0;
  st = vsa_layer_norm_bwd_workspace_size(B, S, x->heads, width, &need);
  if (st != VSA_OK) return st;
  if (workspace_bytes < need) return VSA_ERR_WORKSPACE_TOO_SMALL;
  if (a.R.n == 0) {
    for (float* p : {dweight, dbias}) {
      const cudaError_t e = p ? cudaMemsetAsync(p, 0, static_cast<size_t>(width) * 4, stream) : cudaSuccess;
      if (e != cudaSuccess) return cuda_fail("vsa_layer_norm_bwd: cudaMemsetAsync", e);
    }
    return VSA_OK;
  }
  if (!mean || !rstd) return VSA_ERR_INVALID_ARG;
  a.dy = dy->data;
  a.x = x->data;
  a.w = weight;
  a.w_f32 = weight_dtype == VSA_F32;
  a.w_wide = aligned(weight, 16);
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx->data;
  a.dx_f32 = dx->dtype == VSA_F32;
  a.sdy = view_strides(dy, B, S);
  a.sx = view_strides(x, B, S);
  a.sdx = view_strides(dx, B, S);
  flatten(&a.R, B, S, &a.sdy, &a.sx, &a.sdx);
  a.part = dweight || dbias ? static_cast<float*>(workspace) : nullptr;
  a.width = width;
  a.inv_n = 1.0f / static_cast<float>(width);
  const int vec = 16 / static_cast<int>(dtype_bytes(x->dtype));
  const bool wide = vec_ok(x, a.sx, vec, width) && vec_ok(dy, a.sdy, vec, width) && vec_ok(dx, a.sdx, vec, width);
  const Shape s = shape_of(width, wide ? vec : 1, a.R.n, 1);
  const int n = bwd_blocks(a.R.n, s, device_sms());           // at most those that the workspace was sized for
  const bool g32 = dy->dtype == VSA_F32;
  if (x->dtype == VSA_F32)
    st = wide ? bwd_launch<float, float, 4>(s, a, n, stream) : bwd_launch<float, float, 1>(s, a, n, stream);
  else if (x->dtype == VSA_BF16 && g32)
    st = wide ? bwd_launch<bf16, float, 8>(s, a, n, stream) : bwd_launch<bf16, float, 1>(s, a, n, stream);
  else if (x->dtype == VSA_BF16)
    st = wide ? bwd_launch<bf16, bf16, 8>(s, a, n, stream) : bwd_launch<bf16, bf16, 1>(s, a, n, stream);
  else if (g32)
    st = wide ? bwd_launch<f16, float, 8>(s, a, n, stream) : bwd_launch<f16, float, 1>(s, a, n, stream);
  else
    st = wide ? bwd_launch<f16, f16, 8>(s, a, n, stream) : bwd_launch<f16, f16, 1>(s, a, n, stream);
  if (st != VSA_OK) return st;
  if (!a.part) return VSA_OK;
  const dim3 grid((width + kSumCols - 1) / kSumCols, 2);
  norm_sum_kernel<<<grid, kSumCols * kSumRows, 0, stream>>>(a.part, n, width, dweight, dbias);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK : cuda_fail("vsa_layer_norm_bwd: sums", e);
}

}  // extern "C"

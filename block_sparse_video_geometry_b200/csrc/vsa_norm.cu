// Layer norm over the last dimension, forward and backward with the gradients
// of weight and bias.
//
// Mathematics: m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), xh = (x - m) r,
// y = xh w + b; with g = dy w: dx = r (g - mean(g) - xh mean(g xh)),
// dw = sum_rows dy xh, db = sum_rows dy. The variance is taken about the mean
// from values held in registers (a one-pass E[x^2] - m^2 loses the rows whose
// mean is far from zero).
//
// Bound: HBM (forward: x read, y written; backward: x, dy read, dx written). A
// row is read once into registers, by a group of lanes of one warp when it is
// short and by one block when it is long. Backward: every thread owns fixed
// columns and sums dw and db of the rows its block passes in registers; blocks
// leave one partial row each, which a second kernel adds in a fixed order (no
// atomics: equal inputs give equal bits).

#include <algorithm>
#include <cmath>

#include "vec.cuh"
#include "vsa_internal.h"

namespace vsa {
namespace {

constexpr int kWarpBlock = 256;      // threads of a block of the short-row kernels

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

// ------------------------------------------------------------------ forward
// A row is spread over TPR threads (LANES of a warp, or the block), E vectors of
// VEC elements each: vector i of thread t is i * TPR + t. The row stays packed
// in registers between its passes (sum, squares, output). U rows per group are
// in flight at once.
template <class T, int VEC, int E, int LANES, int U, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const __grid_constant__ FwdArgs a) {
  constexpr bool kWarp = LANES <= 32;
  constexpr int kLanes = kWarp ? LANES : 32;
  __shared__ float red[2][2][32];
  const int tpr = kWarp ? LANES : blockDim.x;
  const int t = kWarp ? threadIdx.x % LANES : threadIdx.x;
  const int groups = kWarp ? kWarpBlock / LANES : 1;
  const int group = kWarp ? threadIdx.x / LANES : 0;
  const int nv = a.width / VEC;
  // A short row's weights stay in registers; a long row's come from L1 with each row.
  constexpr bool kKeep = E * VEC <= 8;
  float w[kKeep ? E : 1][VEC], b[kKeep ? E : 1][VEC];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < E; ++i) weights<T, VEC>(a, i * tpr + t, nv, w[i], b[i]);
  }
  int phase = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups * U;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * groups * U; r0 < a.R.n; r0 += step) {
    Pack<T, VEC> k[U][E];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r0 + u * groups + group;
      if (row >= a.R.n) continue;
      const T* x = static_cast<const T*>(a.x) + offset(a.sx, place(a.R, row));
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i * tpr + t < nv) k[u][i].load(x + static_cast<int64_t>(i * tpr + t) * VEC);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r0 + u * groups + group;
      const bool live = row < a.R.n;               // whole lane groups; every lane takes part in the sums
      float sum = 0.0f, sq = 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (!live || i * tpr + t >= nv) continue;
        float v[VEC];
        k[u][i].get(v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum += v[j];
      }
      const float mean = (kWarp ? lane_sum<kLanes>(sum) : block_sum(sum, red[phase][0])) * a.inv_n;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (!live || i * tpr + t >= nv) continue;
        float v[VEC];
        k[u][i].get(v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) sq = fmaf(v[j] - mean, v[j] - mean, sq);
      }
      const float var = (kWarp ? lane_sum<kLanes>(sq) : block_sum(sq, red[phase][1])) * a.inv_n;
      phase ^= 1;
      const float rstd = 1.0f / sqrtf(var + a.eps);
      if (!live) continue;
      T* y = static_cast<T*>(a.y) + offset(a.sy, place(a.R, row));
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = i * tpr + t;
        if (c >= nv) continue;
        float v[VEC], wl[VEC], bl[VEC];
        if constexpr (!kKeep) weights<T, VEC>(a, c, nv, wl, bl);
        k[u][i].get(v);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          v[j] = fmaf((v[j] - mean) * rstd, kKeep ? w[kKeep ? i : 0][j] : wl[j], kKeep ? b[kKeep ? i : 0][j] : bl[j]);
        k[u][i].set(v);
        k[u][i].store(y + static_cast<int64_t>(c) * VEC);
      }
      if (t == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
      }
    }
  }
}

// ----------------------------------------------------------------- backward
// Same spread. A thread keeps the weights and the running dw and db of its
// columns, and loads the next rows while it works on the current ones.
template <class T, class G, int VEC, int E, int LANES, int U, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const __grid_constant__ BwdArgs a) {
  constexpr bool kWarp = LANES <= 32;
  __shared__ float red[2][2][32];
  const int tpr = kWarp ? LANES : blockDim.x;
  const int t = kWarp ? threadIdx.x % LANES : threadIdx.x;
  const int groups = kWarp ? kWarpBlock / LANES : 1;
  const int group = kWarp ? threadIdx.x / LANES : 0;
  const int nv = a.width / VEC;
  float w[E][VEC], dw[E][VEC], db[E][VEC];
#pragma unroll
  for (int i = 0; i < E; ++i) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] = 1.0f, dw[i][j] = 0.0f, db[i][j] = 0.0f;
    const int c = i * tpr + t;
    if (a.w && c < nv) load_weight<T, VEC>(a.w, a.w_f32, a.w_wide, c * VEC, w[i]);
  }
  Pack<T, VEC> kx[U][E];
  Pack<G, VEC> kg[U][E];
  float mean[U], rstd[U];
  auto fetch = [&](int64_t r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r0 + u * groups + group;
      mean[u] = rstd[u] = 0.0f;
      if (row >= a.R.n) continue;
      const Place p = place(a.R, row);
      const T* x = static_cast<const T*>(a.x) + offset(a.sx, p);
      const G* dy = static_cast<const G*>(a.dy) + offset(a.sdy, p);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int64_t c = i * tpr + t;
        if (c >= nv) continue;
        kx[u][i].load(x + c * VEC);
        kg[u][i].load(dy + c * VEC);
      }
      mean[u] = a.mean[row];
      rstd[u] = a.rstd[row];
    }
  };
  int phase = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups * U;
  int64_t r0 = static_cast<int64_t>(blockIdx.x) * groups * U;
  if (r0 < a.R.n) fetch(r0);
  for (; r0 < a.R.n; r0 += step) {
    // the rows stay packed between the two passes: unpacked they would not fit
    Pack<T, VEC> cx[U][E];
    Pack<G, VEC> cg[U][E];
    float s1[U], s2[U], mu[U], rs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = r0 + u * groups + group < a.R.n;
      s1[u] = s2[u] = 0.0f;
      mu[u] = mean[u];
      rs[u] = rstd[u];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (!live || i * tpr + t >= nv) continue;
        cx[u][i] = kx[u][i];
        cg[u][i] = kg[u][i];
        float xh[VEC], g[VEC];
        cx[u][i].get(xh);
        cg[u][i].get(g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xh[j] = (xh[j] - mu[u]) * rs[u];
          dw[i][j] = fmaf(g[j], xh[j], dw[i][j]);
          db[i][j] += g[j];
          g[j] *= w[i][j];
          s1[u] += g[j];
          s2[u] = fmaf(g[j], xh[j], s2[u]);
        }
      }
    }
    // dx may lie over dy: a row is fetched and written by the same block, in that order
    if (r0 + step < a.R.n) fetch(r0 + step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s1[u] = lane_sum<kWarp ? LANES : 32>(s1[u]);
      s2[u] = lane_sum<kWarp ? LANES : 32>(s2[u]);
    }
    if constexpr (!kWarp) {
      static_assert(U == 1, "one row per block");
      const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
      if (warps > 1) {
        if (lane == 0) {
          red[phase][0][threadIdx.x >> 5] = s1[0];
          red[phase][1][threadIdx.x >> 5] = s2[0];
        }
        __syncthreads();
        s1[0] = lane_sum<32>(lane < warps ? red[phase][0][lane] : 0.0f);
        s2[0] = lane_sum<32>(lane < warps ? red[phase][1][lane] : 0.0f);
        phase ^= 1;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = r0 + u * groups + group;
      if (row >= a.R.n) continue;
      const float c1 = s1[u] * a.inv_n, c2 = s2[u] * a.inv_n;
      const int64_t od = offset(a.sdx, place(a.R, row));
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int c = i * tpr + t;
        if (c >= nv) continue;
        float o[VEC], g[VEC];
        cx[u][i].get(o);
        cg[u][i].get(g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = rs[u] * (g[j] * w[i][j] - fmaf((o[j] - mu[u]) * rs[u], c2, c1));
        const int64_t at = od + static_cast<int64_t>(c) * VEC;
        if (a.dx_f32) {
          Pack<float, VEC> k;
          k.set(o);
          k.store(static_cast<float*>(a.dx) + at);
        } else {
          Pack<T, VEC> k;
          k.set(o);
          k.store(static_cast<T*>(a.dx) + at);
        }
      }
    }
  }
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.width;
  if constexpr (kWarp) {
    // the block's row groups first, in group order
    __shared__ float acc[2][LANES * E * VEC];
    for (int i = threadIdx.x; i < 2 * LANES * E * VEC; i += kWarpBlock) (&acc[0][0])[i] = 0.0f;
    for (int gidx = 0; gidx < kWarpBlock / LANES; ++gidx) {
      __syncthreads();
      if (group != gidx) continue;
#pragma unroll
      for (int i = 0; i < E; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          acc[0][(i * LANES + t) * VEC + j] += dw[i][j];
          acc[1][(i * LANES + t) * VEC + j] += db[i][j];
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.width; c += kWarpBlock) {
      part[c] = acc[0][c];
      part[a.width + c] = acc[1][c];
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = i * tpr + t;
      if (c >= nv) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        part[c * VEC + j] = dw[i][j];
        part[a.width + c * VEC + j] = db[i][j];
      }
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
#pragma unroll 4
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
// block per row with `ept` elements per thread.
struct Shape {
  int vec, lanes;         // lanes 64: one block per row
  int ept;
  int threads, rows_per_block;
};
constexpr int kFwdU = 4, kBwdU = 2;   // rows in flight per lane group of the short-row kernels

Shape shape_of(int width, int vec, int ept, int u) {
  const int nv = width / vec;
  if (nv <= 32) {
    const int lanes = nv <= 16 ? 16 : 32;
    return Shape{vec, lanes, vec, kWarpBlock, kWarpBlock / lanes * u};
  }
  const int e = ept / vec;
  return Shape{vec, 64, ept, ((nv + e - 1) / e + 31) / 32 * 32, 1};
}

// Forward: 32 elements per thread (four 16-byte loads of bf16 in flight) once
// the rows fill the GPU; few rows are spread over more threads.
int fwd_ept(int width, int64_t rows) {
  if (width > 8192) return rows >= 512 ? 32 : 16;
  return rows >= 512 && width >= 2048 ? 32 : 8;
}
// Backward: 16 elements per thread, so that weights, dw, db, two rows and the
// next rows' packed data fit its registers; 8 for narrow rows.
int bwd_ept(int width) { return width > 1024 ? 16 : 8; }

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  return n;
}

constexpr int kMaxSms = 160;                        // the workspace is sized for this many
// Blocks of the backward kernel: a partial row each, so no more than fill the GPU.
int bwd_blocks(int64_t rows, const Shape& s) {
  const int per_sm = std::max(1, std::min(8, 640 / s.threads));
  const int64_t most = static_cast<int64_t>(std::min(sm_count(), kMaxSms)) * per_sm;
  return static_cast<int>(std::min<int64_t>((rows + s.rows_per_block - 1) / s.rows_per_block, most));
}

template <class T, int VEC>
void fwd_launch(const Shape& s, const FwdArgs& a, cudaStream_t stream) {
  const int64_t groups = (a.R.n + s.rows_per_block - 1) / s.rows_per_block;
  const int blocks = static_cast<int>(std::min<int64_t>(groups, 1 << 20));
  if (s.lanes == 16) norm_fwd_kernel<T, VEC, 1, 16, kFwdU, kWarpBlock><<<blocks, s.threads, 0, stream>>>(a);
  else if (s.lanes == 32) norm_fwd_kernel<T, VEC, 1, 32, kFwdU, kWarpBlock><<<blocks, s.threads, 0, stream>>>(a);
  else if (s.ept == 32) norm_fwd_kernel<T, VEC, 32 / VEC, 64, 1, 512><<<blocks, s.threads, 0, stream>>>(a);
  else if (s.ept == 16) norm_fwd_kernel<T, VEC, 16 / VEC, 64, 1, 1024><<<blocks, s.threads, 0, stream>>>(a);
  else norm_fwd_kernel<T, VEC, 8 / VEC, 64, 1, 1024><<<blocks, s.threads, 0, stream>>>(a);
}

template <class T, class G, int VEC>
void bwd_launch(const Shape& s, const BwdArgs& a, int blocks, cudaStream_t stream) {
  if (s.lanes == 16) norm_bwd_kernel<T, G, VEC, 1, 16, kBwdU, kWarpBlock><<<blocks, s.threads, 0, stream>>>(a);
  else if (s.lanes == 32) norm_bwd_kernel<T, G, VEC, 1, 32, kBwdU, kWarpBlock><<<blocks, s.threads, 0, stream>>>(a);
  else if (s.ept == 8) norm_bwd_kernel<T, G, VEC, 8 / VEC, 64, 1, 640><<<blocks, s.threads, 0, stream>>>(a);
  else if (s.threads <= 640) norm_bwd_kernel<T, G, VEC, 16 / VEC, 64, 1, 640><<<blocks, s.threads, 0, stream>>>(a);
  else norm_bwd_kernel<T, G, VEC, 16 / VEC, 64, 1, 1024><<<blocks, s.threads, 0, stream>>>(a);
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
  const Shape s = shape_of(width, wide ? vec : 1, fwd_ept(width, a.R.n), kFwdU);
  if (x->dtype == VSA_F32) wide ? fwd_launch<float, 4>(s, a, stream) : fwd_launch<float, 1>(s, a, stream);
  else if (x->dtype == VSA_BF16) wide ? fwd_launch<bf16, 8>(s, a, stream) : fwd_launch<bf16, 1>(s, a, stream);
  else wide ? fwd_launch<f16, 8>(s, a, stream) : fwd_launch<f16, 1>(s, a, stream);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK : cuda_fail("vsa_layer_norm_fwd", e);
}

vsa_status vsa_layer_norm_bwd_workspace_size(int32_t B, int64_t S, int32_t heads, int32_t width, size_t* bytes) {
  Rows R;
  if (!bytes) return VSA_ERR_INVALID_ARG;
  const vsa_status st = check_rows(B, S, heads, width, &R);
  if (st != VSA_OK) return st;
  // a partial row of dw and db per block: at most 8 blocks per SM
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>(R.n, kMaxSms * 8));
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
  const Shape s = shape_of(width, wide ? vec : 1, bwd_ept(width), kBwdU);
  const int blocks = bwd_blocks(a.R.n, s);
  const bool g32 = dy->dtype == VSA_F32;
  if (x->dtype == VSA_F32) {
    wide ? bwd_launch<float, float, 4>(s, a, blocks, stream) : bwd_launch<float, float, 1>(s, a, blocks, stream);
  } else if (x->dtype == VSA_BF16) {
    if (g32) wide ? bwd_launch<bf16, float, 8>(s, a, blocks, stream) : bwd_launch<bf16, float, 1>(s, a, blocks, stream);
    else wide ? bwd_launch<bf16, bf16, 8>(s, a, blocks, stream) : bwd_launch<bf16, bf16, 1>(s, a, blocks, stream);
  } else {
    if (g32) wide ? bwd_launch<f16, float, 8>(s, a, blocks, stream) : bwd_launch<f16, float, 1>(s, a, blocks, stream);
    else wide ? bwd_launch<f16, f16, 8>(s, a, blocks, stream) : bwd_launch<f16, f16, 1>(s, a, blocks, stream);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail("vsa_layer_norm_bwd", e);
  if (!a.part) return VSA_OK;
  const dim3 grid((width + kSumCols - 1) / kSumCols, 2);
  norm_sum_kernel<<<grid, kSumCols * kSumRows, 0, stream>>>(a.part, blocks, width, dweight, dbias);
  e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK : cuda_fail("vsa_layer_norm_bwd: sums", e);
}

}  // extern "C"

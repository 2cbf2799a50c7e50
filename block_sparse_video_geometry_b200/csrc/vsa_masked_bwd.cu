// Dense attention with capped scores, a distance bias, document and prefix
// masks: backward pass.
//
// Mathematics: P = exp(s - lse) from the forward's lse, D = sum_d dO O,
// dS = P (dO V^T - D) (times 1 - tanh^2 under a cap), dV = P^T dO,
// dK = scale dS^T Q, dQ = scale dS K.
//
// Roundings to bf16: P and dS as operands of the accumulating products (the tensor cores
// take nothing wider at this rate; a sum of many terms is off by a relative 0.0016 from
// it, like one rounding of the result), and `out`, which the caller kept and D is formed
// from (dq and dk 0.0024 without, 0.0027 with it, more for rows of few keys; exact D would
// take two more products per pair). The results are rounded once more. Sums, P, dS, D and
// the statistics are 32-bit.
//
// Bound: tensor pipe. The formulas need five products per visible pair; the two
// kinds of blocks here run seven (S and dO V^T once per side), so that every sum stays
// in one block's TMEM in a fixed order: no atomics, equal inputs give equal bits,
// and dQ needs no 32-bit traffic through memory. Measured: 4096 x 4096, 24 heads 640
// us (1130 TFLOP/s of the seven products), documents packed in 8,192 tokens 850 us.
//
// Design.
//  * dkv_block: a block owns 128 keys of a key head (TMEM lane = key) and walks
//    the query tiles that see them, for every query head of the group:
//    S^T = K Q^T, dP^T = V dO^T, then dV += P^T dO and dK += dS^T Q with P^T and
//    dS^T (bf16) as A operands in TMEM over their own 32-bit columns. Two warps
//    issue products, one S^T and dV, one dP^T and dK; each rewrites its columns
//    behind its own accumulation, in issue order. The two halves of a tile's query
//    columns are pipelines of their own, with barriers of their own. Sixteen warps
//    (four per lane quadrant, 32 query columns each, so two per quadrant and half)
//    turn S^T into P^T while dP^T and dK run, and dP^T into dS^T while dV and the
//    next S^T run.
//  * dq_block: a block owns 128 queries of a head (lane = query) and walks the
//    key tiles: S = Q K^T, dP = dO V^T, dQ += dS K, dS in two buffers of its own.
// Both read their tiles by TMA, three stages of the tensor that is used from the
// scores to the accumulation, two of the other. D and lse in log2 units come from
// prepare_kernel, negated; rows without visible keys get -inf there, so that P = 0.
// Every wait is bounded (see vsa_masked_attn_status).

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "masked_scores.cuh"
#include "sm100.cuh"
#include "vsa_masked.h"

namespace vsa {
namespace masked {
namespace {


// ------------------------------------------------------------------ prepare
// Minus D and minus lse2 of every row, [B][Hq][nqt * 128]; rows past Sq, and rows
// without visible keys: 0 and -inf, so that P = 0. Where the call masks anything,
// also the rows of dout, q and k with an infinity or NaN (see Clean). One block per
// (head of q, then of k; tile) in x and batch entry, heads first: neighbours read
// neighbouring memory. HBM bound: out and dout (and q, k) read once.
struct PrepArgs {
  const uint16_t *out, *dout, *q, *k;
  Strides so, sd, sq, sk;
  const float* lse;
  int32_t Hq, Hk, Sq, Sk, nqt, nkt, masked;
  float *lse2, *delta;
  Clean clean_q, clean_o, clean_k;
};

__device__ __forceinline__ float dot8(uint4 a, uint4 b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
    s = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), s);
  }
  return s;
}

__global__ void __launch_bounds__(kTileThreads, 2) prepare_kernel(const __grid_constant__ PrepArgs a) {
  const int heads = a.Hq + (a.masked ? a.Hk : 0), tile = blockIdx.x / heads, b = blockIdx.y;
  const int head = blockIdx.x % heads;
  const bool key = head >= a.Hq;
  const int h = key ? head - a.Hq : head;
  if (tile >= (key ? a.nkt : a.nqt)) return;               // the whole block
  __shared__ uint32_t bad[2][4];
  if (threadIdx.x < 8) (&bad[0][0])[threadIdx.x] = 0;
  __syncthreads();
  const int64_t r0 = static_cast<int64_t>(tile) * kRows;
  uint4 w[kPieces];
  if (key) {
    load_pieces(w, a.k + b * a.sk.b + r0 * a.sk.s + h * a.sk.h, a.sk.s, min(kRows, a.Sk - tile * kRows));
    find_bad(w, bad[0]);
    __syncthreads();
    write_clean(a.clean_k, w, bad[0], b, h, a.Hk, tile, a.nkt, a.Sk);
    return;
  }
  // all loads of the tile in flight at once
  const int n = min(kRows, a.Sq - tile * kRows);
  uint4 o[kPieces], wq[kPieces];
  load_pieces(w, a.dout + b * a.sd.b + r0 * a.sd.s + h * a.sd.h, a.sd.s, n);
  load_pieces(o, a.out + b * a.so.b + r0 * a.so.s + h * a.so.h, a.so.s, n);
  if (a.masked) load_pieces(wq, a.q + b * a.sq.b + r0 * a.sq.s + h * a.sq.h, a.sq.s, n);
  const size_t row0 = (static_cast<size_t>(b) * a.Hq + h) * a.nqt * kRows + r0;
  if (threadIdx.x < kRows) {
    const int r = threadIdx.x;
    const float l = r < n ? a.lse[(static_cast<size_t>(b) * a.Hq + h) * a.Sq + r0 + r] * -kLog2e : -INFINITY;
    a.lse2[row0 + r] = l == INFINITY ? -INFINITY : l;
  }
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int e = i * kTileThreads + threadIdx.x, r = e >> 4;
    float d = dot8(w[i], o[i]);                            // rows past n: zero
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) d += __shfl_xor_sync(0xffffffffu, d, s);
    if ((e & 15) == 0) a.delta[row0 + r] = -d;
  }
  if (!a.masked) return;
  find_bad(w, bad[0]);
  find_bad(wq, bad[1]);
  __syncthreads();
  write_clean(a.clean_o, w, bad[0], b, h, a.Hq, tile, a.nqt, a.Sq);
  write_clean(a.clean_q, wq, bad[1], b, h, a.Hq, tile, a.nqt, a.Sq);
}

// ------------------------------------------------------------------- shared
constexpr int kThreads = 608;
constexpr int kEw = 16;                      // elementwise warps: four per lane quadrant, 32 columns each
constexpr int kWarpLoad = kEw, kWarpX = kEw + 1, kWarpY = kEw + 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kIdescKK = idesc_bf16_f32(128, 128, 0, 0);   // A and B K-major
constexpr uint32_t kIdescKK64 = idesc_bf16_f32(128, 64, 0, 0);  // 64 rows of B
constexpr uint32_t kIdescKM = idesc_bf16_f32(128, 128, 0, 1);   // A K-major (TMEM), B MN-major

constexpr int kStagesA = 3;

struct Smem {
  uint8_t own[2][kTileBytes];                // dkv: K, V; dq: Q, dO
  uint8_t ring_a[kStagesA][kTileBytes];      // dkv: Q; dq: K (held from the scores to the accumulation)
  uint8_t ring_b[2][kTileBytes];             // dkv: dO; dq: V
  float lse2[2][kRows], delta[2][kRows];     // dkv: of the query tile's rows, negated
  uint64_t own_full, a_full[kStagesA], a_empty[kStagesA], b_full[2], b_empty[2], rows_full[2];
  uint64_t s_full[2], s_done[2], dp_full[2], ds_done[2];   // dkv: per half of the query columns; dq: [0]
  uint64_t acc[2], drain[2];
  uint32_t tmem_base;
  int abort;
};

struct Args {
  Problem p;
  Clean clean_a, clean_b;                    // of ring_a's and ring_b's tensors, or null
  int32_t a_h, a_b, b_h, b_b;                // 1: the map has that dimension, 0: broadcast
  int32_t o1_h, o1_b, o2_h, o2_b;            // the same of the block's own two tensors
  const float *lse2, *delta;                 // [B][Hq][padded], negated
  int32_t padded, nqt;
  const int32_t *count, *list;               // visible tiles of the other side, or null
  uint16_t *out1, *out2;                     // dkv: dk, dv; dq: dq
  int32_t splits;                            // dkv: parts of a key tile's query tiles, one block each
  float* part;                               // [split][dk, dv][B][Hk][nkt * 128][128], or null (splits == 1)
  Strides so1, so2;
  int* err;
};

__device__ __forceinline__ bool bounded_wait(Smem& sm, uint64_t& bar, uint32_t parity, int* err) {
  const bool ok = mbar_wait(smem_u32(&bar), parity, &sm.abort, kTimeoutNs);
  if (!ok) {
    *reinterpret_cast<volatile int*>(err) = VSA_ERR_TIMEOUT;
    *reinterpret_cast<volatile int*>(&sm.abort) = 1;
  }
  return ok;
}
__device__ __forceinline__ bool warp_wait(Smem& sm, uint64_t& bar, uint32_t parity, int* err) {
  if (__all_sync(0xffffffffu, mbar_test_wait(smem_u32(&bar), parity))) return true;
  return __all_sync(0xffffffffu, bounded_wait(sm, bar, parity, err));
}

// D = A B^T over 128 channels, both K-major tiles in shared memory (32 B per K step
// inside a swizzled row, d halves 16 KB apart): all 128 rows of B, or with `half`
// >= 0 the 64 of one half (8 KB apart) into D's columns 64 half.
__device__ __forceinline__ void product_kk(uint32_t d, const uint8_t* x, const uint8_t* y, int half) {
  const uint64_t xd = smem_desc_sw128(smem_u32(x), 16, 1024);
  const uint64_t yd = smem_desc_sw128(smem_u32(y) + 8192 * max(half, 0), 16, 1024);
  const uint32_t to = d + 64 * max(half, 0), idesc = half < 0 ? kIdescKK : kIdescKK64;
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    umma_ss(to, xd + (kk >> 2) * (16384 >> 4) + (kk & 3) * 2, yd + (kk >> 2) * (16384 >> 4) + (kk & 3) * 2, idesc,
            kk > 0 ? 1u : 0u);
}

// D += A B over 64 rows of B from row 64 half (MN-major: 16 rows = 2 KB per K step, d
// halves 16 KB apart); A in TMEM as bf16 pairs, 8 columns per K step.
__device__ __forceinline__ void product_km(uint32_t d, uint32_t x, int second, const uint8_t* y, int half, bool add) {
  const uint64_t yd = smem_desc_sw128(smem_u32(y) + 8192 * half, 16384, 1024);
#pragma unroll
  for (int kk = 0; kk < 4; ++kk)
    umma_ts(d, x + (kk >> 1) * second + (kk & 1) * 8, yd + kk * (2048 >> 4), kIdescKM, add || kk > 0 ? 1u : 0u);
}

__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, int row, int h, int b, uint64_t& bar) {
  const uint32_t d = smem_u32(dst), f = smem_u32(&bar);
  tma_load_4d(d, map, 0, row, h, b, f);
  tma_load_4d(d + kTileBytes / 2, map, 64, row, h, b, f);
}

__device__ __forceinline__ bool any(uint4 m) { return m.x | m.y | m.z | m.w; }

// 32 columns of 32-bit sums times `f` (or zeros) as bf16 into `row` (a row per lane;
// null: none). They go through the warp's 2 KB at `stage`, so that 64 bytes of a
// row are stored together and not 16 of 32 rows at a time.
__device__ __forceinline__ void write_columns(uint32_t taddr, bool have, float f, uint16_t* row, uint8_t* stage) {
  const int lane = threadIdx.x & 31;
  float o[32];
  __syncwarp();
  if (have) {
    tmem_ld32x32f(taddr, o);
    tmem_wait_ld32(o);
  } else {
#pragma unroll
    for (int u = 0; u < 32; ++u) o[u] = 0.0f;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    *reinterpret_cast<uint4*>(stage + lane * 64 + (u ^ (lane >> 1 & 3)) * 16) =
        make_uint4(pack_bf16x2(o[8 * u] * f, o[8 * u + 1] * f), pack_bf16x2(o[8 * u + 2] * f, o[8 * u + 3] * f),
                   pack_bf16x2(o[8 * u + 4] * f, o[8 * u + 5] * f), pack_bf16x2(o[8 * u + 6] * f, o[8 * u + 7] * f));
  __syncwarp();
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int r = it * 8 + (lane >> 2), k = lane & 3;
    uint16_t* to = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), r));
    if (to)
      *reinterpret_cast<uint4*>(to + 8 * k) = *reinterpret_cast<const uint4*>(stage + r * 64 + (k ^ (r >> 1 & 3)) * 16);
  }
}

// 32 columns of 32-bit sums times `f` (or zeros).
__device__ __forceinline__ void write_part(uint32_t taddr, bool have, float f, float* row) {
  float o[32];
  if (have) {
    tmem_ld32x32f(taddr, o);
    tmem_wait_ld32(o);
  } else {
#pragma unroll
    for (int u = 0; u < 32; ++u) o[u] = 0.0f;
  }
#pragma unroll
  for (int u = 0; u < 32; u += 4)
    *reinterpret_cast<float4*>(row + u) = make_float4(o[u] * f, o[u + 1] * f, o[u + 2] * f, o[u + 3] * f);
}

// Barriers and TMEM; `warps` elementwise warps arrive per score buffer.
template <class Init>
__device__ __forceinline__ uint32_t set_up(Smem& sm, int warps, Init init) {
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sm.own_full), 1);
    for (int i = 0; i < kStagesA; ++i) {
      mbar_init(smem_u32(&sm.a_full[i]), 1);
      mbar_init(smem_u32(&sm.a_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.b_full[i]), 1);
      mbar_init(smem_u32(&sm.rows_full[i]), 1);
      mbar_init(smem_u32(&sm.acc[i]), 1);
      mbar_init(smem_u32(&sm.drain[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm.s_full[i]), 1);
      mbar_init(smem_u32(&sm.s_done[i]), warps);
      mbar_init(smem_u32(&sm.dp_full[i]), 1);
      mbar_init(smem_u32(&sm.ds_done[i]), warps);
    }
    init();
    sm.abort = 0;
    fence_mbar_init();
  }
  if ((threadIdx.x >> 5) == kWarpX) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return sm.tmem_base;
}

__device__ __forceinline__ void finish(uint32_t tmem) {
  tc_fence_before();
  __syncthreads();
  if ((threadIdx.x >> 5) == kWarpX) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Scores of 32 columns in place -> P against `ref` (minus lse in log2 units, a pair
// of columns at a time), and into `w` P times the cap's derivative. Without a
// cap a quarter of the exponentials go to the FMA pipe.
template <bool kCap, bool kBias, class Ref>
__device__ __forceinline__ void probabilities(float (&x)[32], float (&w)[32], const ScoreTerms& s, float d0, float dir,
                                              Ref ref) {
  score_args<kCap, kBias>(x, w, s, d0, dir, ref);          // w: tanh
  const uint64_t one = pack_f32x2(1.0f, 1.0f), neg = pack_f32x2(-1.0f, -1.0f);
#pragma unroll
  for (int u = 0; u < 32; u += 2) {
    ex2_pair(x[u], x[u + 1], !kCap && u % 8 == 4);
    if constexpr (kCap) {
      const uint64_t t = pack_f32x2(w[u], w[u + 1]);
      unpack_f32x2(mul_f32x2(pack_f32x2(x[u], x[u + 1]), fma_f32x2(mul_f32x2(t, neg), t, one)), w[u], w[u + 1]);
    } else {
      w[u] = x[u];
      w[u + 1] = x[u + 1];
    }
  }
}

// x = w (x - delta), delta as minus a pair of columns at a time.
template <class Ref>
__device__ __forceinline__ void score_gradients(float (&x)[32], const float (&w)[32], Ref minus_delta) {
#pragma unroll
  for (int u = 0; u < 32; u += 2) {
    const uint64_t d = add_f32x2(pack_f32x2(x[u], x[u + 1]), minus_delta(u));
    unpack_f32x2(mul_f32x2(pack_f32x2(w[u], w[u + 1]), d), x[u], x[u + 1]);
  }
}

// ----------------------------------------------------------------- dK and dV
template <bool kCap, bool kBias>
__device__ __forceinline__ void dkv_block(Smem& sm, int block, const Args& a, const CUtensorMap& map_k,
                                          const CUtensorMap& map_v, const CUtensorMap& map_q, const CUtensorMap& map_o,
                                          const CUtensorMap& map_qc, const CUtensorMap& map_oc) {
  const Problem& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // early key tiles, the longest under a causal mask, first
  const int per = p.Hk * p.B * a.splits, kt = block / per, split = block % per % a.splits;
  const int hk = block % per / a.splits % p.Hk, b = block % per / a.splits / p.Hk;
  const int k0 = kt * kRows;
  const uint32_t tmem = set_up(sm, kEw / 2, [&] {
    mbar_init(smem_u32(&sm.b_empty[0]), 2);                // dO is read by dP^T and by dV
    mbar_init(smem_u32(&sm.b_empty[1]), 2);
  });
  constexpr uint32_t kColS = 0, kColDp = 128, kColDv = 256, kColDk = 384;

  // query tiles: `len` of them for each query head of the group
  const size_t row = static_cast<size_t>(b) * p.nkt + kt;
  const int prefix = p.causal && p.prefix ? p.prefix[b] : 0;
  int first = 0, len = 0;
  if (a.count) {
    len = a.count[row];
  } else {
    if (p.causal && prefix <= k0) first = max(0, k0 - p.off) / kRows;
    len = max(0, a.nqt - first);
  }
  const int32_t* list = a.count ? a.list + row * a.nqt : nullptr;
  // this block's part of them, counted over the group's heads
  const int all = len * p.group, begin = static_cast<int>(static_cast<int64_t>(all) * split / a.splits);
  const int n = static_cast<int>(static_cast<int64_t>(all) * (split + 1) / a.splits) - begin;
  const int h_begin = hk * p.group + (len ? begin / len : 0), idx_begin = len ? begin % len : 0;

  if (warp == kWarpLoad) {
    if (lane == 0) {
      bool ok = true;
      mbar_arrive_expect_tx(smem_u32(&sm.own_full), 2 * kTileBytes);
      load_tile(sm.own[0], &map_k, k0, a.o1_h ? hk : 0, a.o1_b ? b : 0, sm.own_full);
      load_tile(sm.own[1], &map_v, k0, a.o2_h ? hk : 0, a.o2_b ? b : 0, sm.own_full);
      int j = 0, h = h_begin, idx = idx_begin;
      size_t last = 0;                                     // rows of the tile before
      for (; j <= n; ++j, ++idx) {
        if (idx == len) idx = 0, ++h;
        const int sa = j % kStagesA, sb = j & 1;
        if (j >= kStagesA && !(ok = bounded_wait(sm, sm.a_empty[sa], (j / kStagesA - 1) & 1, a.err))) break;
        if (j > 0) {
          // lse and D of tile j - 1 over those of j - 3: that step has ended (its Q stage is free)
          const uint32_t bar = smem_u32(&sm.rows_full[sb ^ 1]);
          mbar_arrive_expect_tx(bar, 2 * kRows * 4);
          bulk_load(smem_u32(sm.lse2[sb ^ 1]), a.lse2 + last, kRows * 4, bar);
          bulk_load(smem_u32(sm.delta[sb ^ 1]), a.delta + last, kRows * 4, bar);
        }
        if (j == n) break;
        const int qt = (list ? list[idx] : first + idx) & kTileMask;
        const size_t tile = (static_cast<size_t>(b) * p.Hq + h) * a.nqt + qt;
        last = (static_cast<size_t>(b) * p.Hq + h) * a.padded + qt * kRows;
        const bool bad_q = a.clean_a.bad && any(a.clean_a.bad[tile]);
        mbar_arrive_expect_tx(smem_u32(&sm.a_full[sa]), kTileBytes);
        load_tile(sm.ring_a[sa], bad_q ? &map_qc : &map_q, qt * kRows, bad_q || a.a_h ? h : 0, bad_q || a.a_b ? b : 0,
                  sm.a_full[sa]);
        if (j >= 2 && !(ok = bounded_wait(sm, sm.b_empty[sb], (j / 2 - 1) & 1, a.err))) {
          ++j;                                             // its Q is in flight; its dO is not
          break;
        }
        const bool bad_o = a.clean_b.bad && any(a.clean_b.bad[tile]);
        mbar_arrive_expect_tx(smem_u32(&sm.b_full[sb]), kTileBytes);
        load_tile(sm.ring_b[sb], bad_o ? &map_oc : &map_o, qt * kRows, bad_o || a.b_h ? h : 0, bad_o || a.b_b ? b : 0,
                  sm.b_full[sb]);
      }
      if (!ok || n == 0) {                                 // every issued copy lands before the block exits
        mbar_wait(smem_u32(&sm.own_full), 0, nullptr, kDrainNs);
        for (int i = max(0, j - 4); i < j; ++i) {
          mbar_wait(smem_u32(&sm.a_full[i % kStagesA]), (i / kStagesA) & 1, nullptr, kDrainNs);
          mbar_wait(smem_u32(&sm.b_full[i & 1]), (i / 2) & 1, nullptr, kDrainNs);
          mbar_wait(smem_u32(&sm.rows_full[i & 1]), (i / 2) & 1, nullptr, kDrainNs);
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpX || warp == kWarpY) {
    // X: S^T (reads Q) and dV (reads dO); Y: dP^T (reads dO) and dK (reads Q). The
    // two halves of the query columns are pipelines of their own: the next scores
    // of a half follow its accumulation, while the other half's warps work. (With
    // all 128 columns at once the elementwise warps waited 1000 of 4150 cycles a
    // step for dV and the next S^T.)
    const bool x = warp == kWarpX;
    if (n > 0) {
      bool ok = warp_wait(sm, sm.own_full, 0, a.err);
      auto q_stage = [&](int j) { return sm.ring_a[j % kStagesA]; };
      auto o_stage = [&](int j) { return sm.ring_b[j & 1]; };
      auto landed = [&](bool q, int j) {
        return q ? warp_wait(sm, sm.a_full[j % kStagesA], (j / kStagesA) & 1, a.err)
                 : warp_wait(sm, sm.b_full[j & 1], (j / 2) & 1, a.err);
      };
      const uint32_t ts = tmem + (x ? kColS : kColDp), to = tmem + (x ? kColDv : kColDk);
      auto scores = [&](int j, int half) {
        if (half == 0 && !landed(x, j)) return false;
        tc_fence_after();
        if (elect_one()) {
          product_kk(ts, sm.own[x ? 0 : 1], x ? q_stage(j) : o_stage(j), half);
          umma_commit(smem_u32(x ? &sm.s_full[half] : &sm.dp_full[half]));
          if (!x && half == 1) umma_commit(smem_u32(&sm.b_empty[j & 1]));
        }
        __syncwarp();
        return true;
      };
      if (ok) ok = scores(0, 0) && scores(0, 1);
      for (int j = 0; ok && j < n; ++j) {
        if (!(ok = landed(!x, j))) break;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (!(ok = warp_wait(sm, x ? sm.s_done[half] : sm.ds_done[half], j & 1, a.err))) break;
          tc_fence_after();
          if (elect_one()) {
            product_km(to, ts + 64 * half, 32, x ? o_stage(j) : q_stage(j), half, j > 0 || half > 0);
            if (half == 1) umma_commit(smem_u32(x ? &sm.b_empty[j & 1] : &sm.a_empty[j % kStagesA]));
            if (half == 1 && j + 1 == n) umma_commit(smem_u32(&sm.acc[x ? 0 : 1]));
          }
          __syncwarp();
          if (j + 1 < n && !(ok = scores(j + 1, half))) break;
        }
      }
      if (!ok && elect_one()) {
        umma_commit(smem_u32(&sm.drain[x ? 0 : 1]));
        mbar_wait(smem_u32(&sm.drain[x ? 0 : 1]), 0, nullptr, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp < kEw) {
    const int quad = warp & 3, part = warp >> 2, half = part >> 1;   // query columns [32 part, + 32)
    const int key = k0 + quad * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t ts = lane_addr + kColS + 32 * part, tp = lane_addr + kColDp + 32 * part;
    ScoreTerms terms(p.scale, p.cap, 0.0f);
    // first query that sees this key by order
    const int i_min = !p.causal || key < prefix ? INT32_MIN : key - p.off;
    const int doc = p.documents && key < p.Sk ? p.doc_k[b * p.doc_k_sb + key] : -1;
    const int32_t* dq = p.documents ? p.doc_q + b * p.doc_q_sb : nullptr;
    bool ok = true;
    int h = h_begin, idx = idx_begin;
    for (int j = 0; j < n; ++j, ++idx) {
      if (idx == len) idx = 0, ++h;
      const int st = j & 1;
      const int rec = list ? list[idx] : first + idx;
      const int qt = rec & kTileMask, q0 = qt * kRows, i0 = q0 + 32 * part;
      // a tile of one document is hidden from a key as a whole or not at all
      const bool by_doc = rec & kPartial0, part_doc = by_doc && !(rec & kOneDoc);
      const bool partial = by_doc || (p.causal && prefix < k0 + kRows && q0 + p.off < k0 + kRows - 1);
      uint32_t bad = 0;                                    // columns whose q or dout holds an infinity or NaN
      if (a.clean_a.bad) {
        const size_t tile = (static_cast<size_t>(b) * p.Hq + h) * a.nqt + qt;
        bad = reinterpret_cast<const uint32_t*>(a.clean_a.bad + tile)[part] |
              reinterpret_cast<const uint32_t*>(a.clean_b.bad + tile)[part];
      }
      if constexpr (kBias) terms.slope = p.slopes[h] * kLog2e;
      // visible columns as a bit mask; only where some pair is hidden
      uint32_t see = 0xffffffffu;
      if (partial) {
        see = 0;
        const int from = by_doc && !part_doc && (doc < 0 || __ldg(dq + q0) != doc) ? INT32_MAX : i_min;
#pragma unroll
        for (int u = 0; u < 32; ++u) see |= (i0 + u >= from ? 1u : 0u) << u;
        if (part_doc) {
#pragma unroll
          for (int u = 0; u < 32; ++u) {
            const int d = __ldg(dq + min(i0 + u, p.Sq - 1));
            if (!(d == doc && d >= 0)) see &= ~(1u << u);
          }
        }
      }
      if (!(ok = warp_wait(sm, sm.rows_full[st], (j / 2) & 1, a.err))) break;
      if (!(ok = warp_wait(sm, sm.s_full[half], j & 1, a.err))) break;
      tc_fence_after();
      float x[32], w[32];
      uint32_t pw[16];
      tmem_ld32x32f(ts, x);
      tmem_wait_ld32(x);
      const float* lse = sm.lse2[st] + 32 * part;
      probabilities<kCap, kBias>(x, w, terms, static_cast<float>(i0 + p.off - key), 1.0f,
                                 [&](int u) { return *reinterpret_cast<const uint64_t*>(lse + u); });
      if (partial) {
#pragma unroll
        for (int u = 0; u < 32; ++u) x[u] = (see >> u) & 1u ? x[u] : 0.0f;
      }
      if (bad) {
#pragma unroll
        for (int u = 0; u < 32; ++u)
          if ((bad & see) >> u & 1u) x[u] = w[u] = NAN;
      }
#pragma unroll
      for (int u = 0; u < 16; ++u) pw[u] = pack_bf16x2(x[2 * u], x[2 * u + 1]);
      tmem_st32x16(ts, pw);                                // over this warp's own columns
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.s_done[half]));
      if (!(ok = warp_wait(sm, sm.dp_full[half], j & 1, a.err))) break;
      tc_fence_after();
      tmem_ld32x32f(tp, x);
      tmem_wait_ld32(x);
      const float* dl = sm.delta[st] + 32 * part;
      score_gradients(x, w, [&](int u) { return *reinterpret_cast<const uint64_t*>(dl + u); });
      if (partial) {
#pragma unroll
        for (int u = 0; u < 32; ++u) x[u] = (see >> u) & 1u ? x[u] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 16; ++u) pw[u] = pack_bf16x2(x[2 * u], x[2 * u + 1]);
      tmem_st32x16(tp, pw);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.ds_done[half]));
    }
    if (ok) {                                              // K and V are read no more; nor are they on their way
      ok = n > 0 ? warp_wait(sm, sm.acc[0], 0, a.err) && warp_wait(sm, sm.acc[1], 0, a.err)
                 : warp_wait(sm, sm.own_full, 0, a.err);
      tc_fence_after();
    }
    if (ok && a.part) {
      const size_t rows = static_cast<size_t>(p.B) * p.Hk * p.nkt * kRows;
      const size_t at = (static_cast<size_t>(b) * p.Hk + hk) * p.nkt * kRows + key;
      float* dst = a.part + (2 * split * rows + at) * kHeadDim + 32 * part;
      write_part(lane_addr + kColDk + 32 * part, n > 0, p.scale, dst);
      write_part(lane_addr + kColDv + 32 * part, n > 0, 1.0f, dst + rows * kHeadDim);
    } else if (ok) {
      const bool live = key < p.Sk;
      const int64_t kk = live ? key : 0;
      write_columns(lane_addr + kColDk + 32 * part, n > 0, p.scale,
                    live ? a.out1 + b * a.so1.b + kk * a.so1.s + hk * a.so1.h + 32 * part : nullptr,
                    sm.own[0] + warp * 2048);
      write_columns(lane_addr + kColDv + 32 * part, n > 0, 1.0f,
                    live ? a.out2 + b * a.so2.b + kk * a.so2.s + hk * a.so2.h + 32 * part : nullptr,
                    sm.own[1] + warp * 2048);
    }
  }
  finish(tmem);
}

// ------------------------------------------------------------------------ dQ
template <bool kCap, bool kBias>
__device__ __forceinline__ void dq_block(Smem& sm, int block, const Args& a, const CUtensorMap& map_q,
                                         const CUtensorMap& map_o, const CUtensorMap& map_k, const CUtensorMap& map_v,
                                         const CUtensorMap& map_kc) {
  const Problem& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = p.Hq * p.B, qt = a.nqt - 1 - block / per;   // late query tiles first
  const int h = block % per % p.Hq, b = block % per / p.Hq, hk = h / p.group;
  const int q0 = qt * kRows;
  const uint32_t tmem = set_up(sm, kEw, [&] {
    mbar_init(smem_u32(&sm.b_empty[0]), 1);
    mbar_init(smem_u32(&sm.b_empty[1]), 1);
  });
  constexpr uint32_t kColS = 0, kColDp = 128, kColDq = 256, kColDs = 384;   // dS: two buffers of 64 columns

  const size_t row = static_cast<size_t>(b) * a.nqt + qt;
  const int n = a.count ? a.count[row] : max(0, p.limit(b, min(q0 + kRows, p.Sq) - 1) + kRows) / kRows;
  const int32_t* list = a.count ? a.list + row * p.nkt : nullptr;
  const uint4* bad = a.clean_a.bad ? a.clean_a.bad + (static_cast<size_t>(b) * p.Hk + hk) * p.nkt : nullptr;

  if (warp == kWarpLoad) {
    if (lane == 0) {
      bool ok = true;
      mbar_arrive_expect_tx(smem_u32(&sm.own_full), 2 * kTileBytes);
      load_tile(sm.own[0], &map_q, q0, a.o1_h ? h : 0, a.o1_b ? b : 0, sm.own_full);
      load_tile(sm.own[1], &map_o, q0, a.o2_h ? h : 0, a.o2_b ? b : 0, sm.own_full);
      int j = 0;
      for (; ok && j < n; ++j) {
        const int st = j & 1, sa = j % kStagesA, kt = (list ? list[j] : j) & kTileMask;
        if (j >= 2 && !(ok = bounded_wait(sm, sm.b_empty[st], (j / 2 - 1) & 1, a.err))) break;
        mbar_arrive_expect_tx(smem_u32(&sm.b_full[st]), kTileBytes);
        load_tile(sm.ring_b[st], &map_v, kt * kRows, a.b_h ? hk : 0, a.b_b ? b : 0, sm.b_full[st]);
        if (j >= kStagesA && !(ok = bounded_wait(sm, sm.a_empty[sa], (j / kStagesA - 1) & 1, a.err))) {
          ++j;
          break;
        }
        const bool bad_k = bad && any(bad[kt]);
        mbar_arrive_expect_tx(smem_u32(&sm.a_full[sa]), kTileBytes);
        load_tile(sm.ring_a[sa], bad_k ? &map_kc : &map_k, kt * kRows, bad_k || a.a_h ? hk : 0,
                  bad_k || a.a_b ? b : 0, sm.a_full[sa]);
      }
      if (!ok || n == 0) {
        mbar_wait(smem_u32(&sm.own_full), 0, nullptr, kDrainNs);
        for (int i = max(0, j - 4); i < j; ++i) {
          mbar_wait(smem_u32(&sm.a_full[i % kStagesA]), (i / kStagesA) & 1, nullptr, kDrainNs);
          mbar_wait(smem_u32(&sm.b_full[i & 1]), (i / 2) & 1, nullptr, kDrainNs);
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpX) {
    if (n > 0) {
      bool ok = warp_wait(sm, sm.own_full, 0, a.err);
      for (int j = 0; ok && j < n; ++j) {
        if (!(ok = warp_wait(sm, sm.a_full[j % kStagesA], (j / kStagesA) & 1, a.err))) break;
        if (j > 0 && !(ok = warp_wait(sm, sm.s_done[0], (j - 1) & 1, a.err))) break;    // S(j - 1) was read
        tc_fence_after();
        if (elect_one()) {
          product_kk(tmem + kColS, sm.own[0], sm.ring_a[j % kStagesA], -1);
          umma_commit(smem_u32(&sm.s_full[0]));
        }
        __syncwarp();
      }
      if (!ok && elect_one()) {
        umma_commit(smem_u32(&sm.drain[0]));
        mbar_wait(smem_u32(&sm.drain[0]), 0, nullptr, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == kWarpY) {
    if (n > 0) {
      bool ok = warp_wait(sm, sm.own_full, 0, a.err);
      auto dp = [&](int j) {
        if (!warp_wait(sm, sm.b_full[j & 1], (j / 2) & 1, a.err)) return false;
        tc_fence_after();
        if (elect_one()) {
          product_kk(tmem + kColDp, sm.own[1], sm.ring_b[j & 1], -1);
          umma_commit(smem_u32(&sm.dp_full[0]));
          umma_commit(smem_u32(&sm.b_empty[j & 1]));
        }
        __syncwarp();
        return true;
      };
      if (ok) ok = dp(0);
      for (int j = 0; ok && j < n; ++j) {
        // dS(j) written means dP(j) read; dP(j + 1) goes first, so that the next
        // elementwise step waits for one product only
        if (!(ok = warp_wait(sm, sm.ds_done[0], j & 1, a.err))) break;
        tc_fence_after();
        if (j + 1 < n && !(ok = dp(j + 1))) break;
        if (!(ok = warp_wait(sm, sm.a_full[j % kStagesA], (j / kStagesA) & 1, a.err))) break;
        if (elect_one()) {
          const uint32_t ds = tmem + kColDs + 64 * (j & 1);
          product_km(tmem + kColDq, ds, 16, sm.ring_a[j % kStagesA], 0, j > 0);
          product_km(tmem + kColDq, ds + 32, 16, sm.ring_a[j % kStagesA], 1, true);
          umma_commit(smem_u32(&sm.a_empty[j % kStagesA]));
          if (j + 1 == n) umma_commit(smem_u32(&sm.acc[0]));
        }
        __syncwarp();
      }
      if (!ok && elect_one()) {
        umma_commit(smem_u32(&sm.drain[1]));
        mbar_wait(smem_u32(&sm.drain[1]), 0, nullptr, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp < kEw) {
    const int quad = warp & 3, part = warp >> 2;           // key columns [32 part, + 32)
    const int i_q = min(q0 + quad * 32 + lane, p.Sq - 1);
    const bool live = q0 + quad * 32 + lane < p.Sq;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t ts = lane_addr + kColS + 32 * part, tp = lane_addr + kColDp + 32 * part;
    const size_t at = (static_cast<size_t>(b) * p.Hq + h) * a.padded + q0 + quad * 32 + lane;
    const uint64_t lse2 = pack_f32x2(a.lse2[at], a.lse2[at]), minus_delta = pack_f32x2(a.delta[at], a.delta[at]);
    const ScoreTerms terms(p.scale, p.cap, kBias ? p.slopes[h] : 0.0f);
    const int lim = p.limit(b, i_q), lim0 = p.limit(b, q0);
    const int doc = p.documents && live ? p.doc_q[b * p.doc_q_sb + i_q] : -1;
    const int32_t* dk = p.documents ? p.doc_k + b * p.doc_k_sb : nullptr;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int rec = list ? list[j] : j;
      const int kt = rec & kTileMask, k0 = kt * kRows, col = k0 + 32 * part;
      // a tile of one document is hidden from a row as a whole or not at all
      const bool by_doc = rec & kPartial0, part_doc = by_doc && !(rec & kOneDoc);
      const bool partial = by_doc || k0 + kRows - 1 > lim0;
      const int lim_t = by_doc && !part_doc && (doc < 0 || __ldg(dk + k0) != doc) ? -1 : lim;
      uint32_t bad_k = 0;                                  // columns whose k holds an infinity or NaN
      if (bad) bad_k = reinterpret_cast<const uint32_t*>(bad + kt)[part];
      uint32_t see = 0xffffffffu;
      if (partial) {
        see = 0;
#pragma unroll
        for (int u = 0; u < 32; ++u) see |= (col + u <= lim_t ? 1u : 0u) << u;
        if (part_doc) {
#pragma unroll
          for (int u = 0; u < 32; ++u) {
            const int d = __ldg(dk + min(col + u, p.Sk - 1));
            if (!(d == doc && d >= 0)) see &= ~(1u << u);
          }
        }
      }
      if (!(ok = warp_wait(sm, sm.s_full[0], j & 1, a.err))) break;
      tc_fence_after();
      float x[32], w[32];
      uint32_t pw[16];
      tmem_ld32x32f(ts, x);
      tmem_wait_ld32(x);
      tc_fence_before();                                   // S(j) is in registers: S(j + 1) may replace it
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.s_done[0]));
      probabilities<kCap, kBias>(x, w, terms, static_cast<float>(i_q + p.off - col), -1.0f,
                                 [&](int) { return lse2; });
      if (!(ok = warp_wait(sm, sm.dp_full[0], j & 1, a.err))) break;
      tc_fence_after();
      tmem_ld32x32f(tp, x);
      tmem_wait_ld32(x);
      score_gradients(x, w, [&](int) { return minus_delta; });
      if (partial) {
#pragma unroll
        for (int u = 0; u < 32; ++u) x[u] = (see >> u) & 1u ? x[u] : 0.0f;
      }
      if (bad_k) {
#pragma unroll
        for (int u = 0; u < 32; ++u)
          if ((bad_k & see) >> u & 1u) x[u] = NAN;
      }
#pragma unroll
      for (int u = 0; u < 16; ++u) pw[u] = pack_bf16x2(x[2 * u], x[2 * u + 1]);
      tmem_st32x16(lane_addr + kColDs + 64 * (j & 1) + 16 * part, pw);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.ds_done[0]));
    }
    if (ok) {                                              // Q and dO are read no more; nor are they on their way
      ok = warp_wait(sm, n > 0 ? sm.acc[0] : sm.own_full, 0, a.err);
      tc_fence_after();
    }
    if (ok)
      write_columns(lane_addr + kColDq + 32 * part, n > 0, p.scale,
                    live ? a.out1 + b * a.so1.b + i_q * a.so1.s + h * a.so1.h + 32 * part : nullptr,
                    sm.own[0] + warp * 2048);
  }
  finish(tmem);
}

// Blocks of dK and dV, then blocks of dQ in the same grid: these do not read those,
// and fill the SMs as the last of them end (two kernels: 4096 x
// 24 heads 705 us, so 650; packed documents 886 and 861).
struct Maps {
  CUtensorMap q, k, v, o, qc, oc, kc;
};

template <bool kCap, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
masked_bwd_kernel(const __grid_constant__ Args kv, const __grid_constant__ Args q, const __grid_constant__ Maps m,
                  int n_dkv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {          // swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicExch(kv.err, VSA_ERR_UNSUPPORTED);
    return;
  }
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const int block = blockIdx.x;
  if (block < n_dkv)
    dkv_block<kCap, kBias>(sm, block, kv, m.k, m.v, m.q, m.o, m.qc, m.oc);
  else
    dq_block<kCap, kBias>(sm, block - n_dkv, q, m.q, m.o, m.k, m.v, m.kc);
}

// dk and dv from the blocks' parts, added in order: one piece of 4 channels a thread.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a) {
  const Problem& p = a.p;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, c = e & 31, r = e >> 5;
  if (r >= static_cast<int64_t>(p.B) * p.Sk * p.Hk) return;
  const int64_t h = r % p.Hk, s = r / p.Hk % p.Sk, b = r / p.Hk / p.Sk;
  const size_t rows = static_cast<size_t>(p.B) * p.Hk * p.nkt * kRows;
  const float* src = a.part + (blockIdx.y * rows + (static_cast<size_t>(b) * p.Hk + h) * p.nkt * kRows + s) * kHeadDim + c * 4;
  float4 x = *reinterpret_cast<const float4*>(src);
  for (int i = 1; i < a.splits; ++i) {
    const float4 y = *reinterpret_cast<const float4*>(src + 2 * i * rows * kHeadDim);
    x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
  }
  const Strides st = blockIdx.y ? a.so2 : a.so1;
  *reinterpret_cast<uint2*>((blockIdx.y ? a.out2 : a.out1) + b * st.b + s * st.s + h * st.h + c * 4) =
      make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

// Zeros of [B, S, heads, 128] (no keys, or no queries).
__global__ void __launch_bounds__(256) zero_kernel(uint16_t* x, Strides st, int S, int heads, int64_t n) {
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;   // 16-byte piece
  if (e >= n) return;
  const int64_t r = e >> 4, h = r % heads, t = r / heads;
  *reinterpret_cast<uint4*>(x + t / S * st.b + t % S * st.s + h * st.h + (e & 15) * 8) = make_uint4(0, 0, 0, 0);
}

void zero(const vsa_view* v, int32_t B, int32_t S, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(B) * S * v->heads * 16;
  if (n)
    zero_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(static_cast<uint16_t*>(v->data),
                                                                            view_strides(v, B, S), S, v->heads, n);
}

// Parts of a key tile's query tiles: where the longest block would outlast the rest
// (a causal mask, shared heads, few tiles). Cost in steps of dK and dV (3 us at most): a
// step of dQ is two thirds of one, a block's start and end two. The grid ends with its
// longest block or with all work spread over the SMs and a part of a block's length
// behind it; parts cost their blocks' ends, the traffic of their 32-bit sums and one more
// launch. Measured, us, chosen first: 2 x 1,555 causal tokens, 8 heads on 4: one part 101,
// two 115; 3,000 causal, 9 heads on 3: two 141, one 209, three 149; 6,000 causal, 3 heads
// on 1: three 133, one 285, four 137; 4,000 x 2 heads, no mask: one 90, two 110.
int splits_of(const Problem& p) {
  constexpr double kDq = 2.0 / 3.0;
  const double pairs = static_cast<double>(p.B) * p.Hk, sms = device_sms();
  const int nqt = tiles(p.Sq);
  double total = 0.0, longest = 0.0;
  for (int kt = 0; kt < p.nkt; ++kt) {
    const int first = p.causal ? std::min(nqt, std::max(0, kt * kRows - p.off) / kRows) : 0;
    total += (nqt - first) * p.group;
    longest = std::max(longest, static_cast<double>(nqt - first) * p.group);
  }
  const double dq = kDq * p.nkt + 2.0;                     // the longest block of dQ
  int best = 1;
  double least = 1e300;
  for (int s = 1; s <= 8 && s <= std::max(1.0, longest / 2); ++s) {
    const double part = std::ceil(longest / s) + 2.0;
    const double spread = pairs * (total * (1.0 + kDq) + 2.0 * p.nkt * s + 2.0 * nqt * p.group) / sms + 0.3 * dq;
    double t = std::max(std::max(part, dq), spread);
    if (s > 1) t += 2.0 + pairs * p.nkt * kRows * s * 2048.0 / 6.5e12 / 3e-6;
    if (t < least * 0.95) {
      least = t;
      best = s;
    }
  }
  return best;
}

struct Workspace {
  size_t part, lse2, delta, range, range_q, count_q, list_q, count_k, list_k;
  size_t bad_q, bad_o, bad_k, copy_q, copy_o, copy_k, total;
};

Workspace workspace_of(const Problem& p, int splits) {
  Workspace w{};
  size_t off = kHeader;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  const size_t b = static_cast<size_t>(p.B), nkt = static_cast<size_t>(p.nkt), nqt = static_cast<size_t>(tiles(p.Sq));
  if (splits > 1) w.part = take(2 * static_cast<size_t>(splits) * b * p.Hk * nkt * kRows * kHeadDim * sizeof(float));
  w.lse2 = take(b * p.Hq * nqt * kRows * sizeof(float));
  w.delta = take(b * p.Hq * nqt * kRows * sizeof(float));
  if (p.documents) {
    w.range = take(b * nkt * sizeof(int4));
    w.range_q = take(b * nqt * sizeof(int4));
    w.count_q = take(b * nqt * sizeof(int32_t));
    w.list_q = take(b * nqt * nkt * sizeof(int32_t));
    w.count_k = take(b * nkt * sizeof(int32_t));
    w.list_k = take(b * nkt * nqt * sizeof(int32_t));
  }
  if (p.masked) {
    w.bad_q = take(b * p.Hq * nqt * sizeof(uint4));
    w.bad_o = take(b * p.Hq * nqt * sizeof(uint4));
    w.bad_k = take(b * p.Hk * nkt * sizeof(uint4));
    w.copy_q = take(b * p.Sq * p.Hq * kHeadDim * 2);
    w.copy_o = take(b * p.Sq * p.Hq * kHeadDim * 2);
    w.copy_k = take(b * p.Sk * p.Hk * kHeadDim * 2);
  }
  w.total = off;
  return w;
}

template <bool kCap, bool kBias>
vsa_status launch(const Args& dkv, const Args& dq, const Maps& m, cudaStream_t stream) {
  const auto kernel = masked_bwd_kernel<kCap, kBias>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem));
  if (e != cudaSuccess) return cuda_fail("vsa_masked_attn_bwd: shared memory", e);
  const Problem& p = dkv.p;
  const int n_dkv = p.nkt * p.Hk * p.B * dkv.splits;
  kernel<<<n_dkv + dq.nqt * p.Hq * p.B, kThreads, sizeof(Smem), stream>>>(dkv, dq, m, n_dkv);
  if ((e = cudaGetLastError()) != cudaSuccess) return cuda_fail("vsa_masked_attn_bwd", e);
  if (dkv.splits > 1) {
    const int64_t pieces = static_cast<int64_t>(p.B) * p.Sk * p.Hk * (kHeadDim / 4);
    join_kernel<<<dim3(static_cast<unsigned>((pieces + 255) / 256), 2), 256, 0, stream>>>(dkv);
  }
  e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK : cuda_fail("vsa_masked_attn_bwd", e);
}

}  // namespace
}  // namespace masked
}  // namespace vsa

using namespace vsa;
using namespace vsa::masked;

extern "C" {

vsa_status vsa_masked_attn_bwd_workspace_size(const vsa_mask* mask, int32_t B, int32_t Sq, int32_t Sk, int32_t Hq,
                                              int32_t Hk, size_t* bytes) {
  if (!bytes || !mask || (mask->documents != 0 && mask->documents != 1)) return VSA_ERR_INVALID_ARG;
  Problem p;
  vsa_mask m = *mask;
  m.documents = 0;                                        // the tensors are not at hand yet
  const vsa_status st = check(&m, nullptr, B, Sq, Sk, Hq, Hk, &p);
  if (st != VSA_OK) return st;
  p.documents = mask->documents;
  p.masked |= mask->documents;
  *bytes = workspace_of(p, splits_of(p)).total;
  return VSA_OK;
}

vsa_status vsa_masked_attn_bwd(const vsa_mask* mask, const vsa_mask_terms* terms, int32_t B, int32_t Sq, int32_t Sk,
                               const vsa_view* q, const vsa_view* k, const vsa_view* v, const vsa_view* out,
                               const float* lse, const vsa_view* dout, const vsa_view* dq, const vsa_view* dk,
                               const vsa_view* dv, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !k || !v || !out || !dout || !dq || !dk || !dv) return VSA_ERR_INVALID_ARG;
  Problem p;
  vsa_status st = check(mask, terms, B, Sq, Sk, q->heads, k->heads, &p);
  for (const vsa_view* x : {q, out, dout})
    if (st == VSA_OK) st = check_tensor(x, B, Sq, q->heads, false);
  for (const vsa_view* x : {k, v})
    if (st == VSA_OK) st = check_tensor(x, B, Sk, k->heads, false);
  if (st == VSA_OK) st = check_tensor(dq, B, Sq, q->heads, true);
  for (const vsa_view* x : {dk, dv})
    if (st == VSA_OK) st = check_tensor(x, B, Sk, k->heads, true);
  if (st != VSA_OK) return st;
  if (reinterpret_cast<uintptr_t>(lse) % 4) return VSA_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256) return VSA_ERR_INVALID_ARG;
  const int splits = splits_of(p);
  const Workspace w = workspace_of(p, splits);
  if (workspace_bytes < w.total) return VSA_ERR_WORKSPACE_TOO_SMALL;
  char* ws = static_cast<char*>(workspace);
  cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), stream);   // this call's status word
  if (e != cudaSuccess) return cuda_fail("vsa_masked_attn_bwd: cudaMemsetAsync", e);
  if (B == 0 || Sq == 0 || Sk == 0) {
    zero(dq, B, Sq, stream);
    zero(dk, B, Sk, stream);
    zero(dv, B, Sk, stream);
    e = cudaGetLastError();
    return e == cudaSuccess ? VSA_OK : cuda_fail("vsa_masked_attn_bwd", e);
  }
  if (!lse) return VSA_ERR_INVALID_ARG;

  Maps m;
  if ((st = make_map(&m.q, q, B, Sq)) != VSA_OK || (st = make_map(&m.k, k, B, Sk)) != VSA_OK ||
      (st = make_map(&m.v, v, B, Sk)) != VSA_OK || (st = make_map(&m.o, dout, B, Sq)) != VSA_OK)
    return st;
  m.qc = m.q;
  m.oc = m.o;
  m.kc = m.k;
  const int nqt = tiles(Sq);
  PrepArgs pa{};
  pa.out = static_cast<const uint16_t*>(out->data);
  pa.dout = static_cast<const uint16_t*>(dout->data);
  pa.q = static_cast<const uint16_t*>(q->data);
  pa.k = static_cast<const uint16_t*>(k->data);
  pa.so = view_strides(out, B, Sq);
  pa.sd = view_strides(dout, B, Sq);
  pa.sq = view_strides(q, B, Sq);
  pa.sk = view_strides(k, B, Sk);
  pa.lse = lse;
  pa.Hq = p.Hq;
  pa.Hk = p.Hk;
  pa.Sq = Sq;
  pa.Sk = Sk;
  pa.nqt = nqt;
  pa.nkt = p.nkt;
  pa.masked = p.masked;
  pa.lse2 = reinterpret_cast<float*>(ws + w.lse2);
  pa.delta = reinterpret_cast<float*>(ws + w.delta);
  if (p.masked) {
    pa.clean_q = Clean{reinterpret_cast<uint4*>(ws + w.bad_q), reinterpret_cast<uint16_t*>(ws + w.copy_q)};
    pa.clean_o = Clean{reinterpret_cast<uint4*>(ws + w.bad_o), reinterpret_cast<uint16_t*>(ws + w.copy_o)};
    pa.clean_k = Clean{reinterpret_cast<uint4*>(ws + w.bad_k), reinterpret_cast<uint16_t*>(ws + w.copy_k)};
    if ((st = make_map(&m.qc, pa.clean_q.copy, B, Sq, p.Hq)) != VSA_OK ||
        (st = make_map(&m.oc, pa.clean_o.copy, B, Sq, p.Hq)) != VSA_OK ||
        (st = make_map(&m.kc, pa.clean_k.copy, B, Sk, p.Hk)) != VSA_OK)
      return st;
  }
  prepare_kernel<<<dim3((p.Hq + (p.masked ? p.Hk : 0)) * (p.masked ? std::max(nqt, p.nkt) : nqt), B), kTileThreads, 0,
                   stream>>>(pa);

  Args g{};
  g.p = p;
  g.lse2 = pa.lse2;
  g.delta = pa.delta;
  g.padded = nqt * kRows;
  g.nqt = nqt;
  g.err = reinterpret_cast<int*>(ws);
  const Strides sq = pa.sq, sd = pa.sd, sk = pa.sk, sv = view_strides(v, B, Sk);
  Args kv = g, qq = g;
  kv.a_h = qq.o1_h = sq.h != 0;
  kv.a_b = qq.o1_b = sq.b != 0;
  kv.b_h = qq.o2_h = sd.h != 0;
  kv.b_b = qq.o2_b = sd.b != 0;
  kv.o1_h = qq.a_h = sk.h != 0;
  kv.o1_b = qq.a_b = sk.b != 0;
  kv.o2_h = qq.b_h = sv.h != 0;
  kv.o2_b = qq.b_b = sv.b != 0;
  kv.out1 = static_cast<uint16_t*>(dk->data);
  kv.so1 = view_strides(dk, B, Sk);
  kv.out2 = static_cast<uint16_t*>(dv->data);
  kv.so2 = view_strides(dv, B, Sk);
  qq.out1 = static_cast<uint16_t*>(dq->data);
  qq.so1 = view_strides(dq, B, Sq);
  if (p.documents) {
    int4* range = reinterpret_cast<int4*>(ws + w.range);
    int32_t *cq = reinterpret_cast<int32_t*>(ws + w.count_q), *lq = reinterpret_cast<int32_t*>(ws + w.list_q);
    int32_t *ck = reinterpret_cast<int32_t*>(ws + w.count_k), *lk = reinterpret_cast<int32_t*>(ws + w.list_k);
    plan(p, kPlanSingle, nqt, range, cq, lq, stream);
    plan_keys(p, range, reinterpret_cast<int4*>(ws + w.range_q), ck, lk, stream);
    qq.count = cq;
    qq.list = lq;
    kv.count = ck;
    kv.list = lk;
  }
  e = cudaGetLastError();                                 // nothing reads sums or lists that nobody wrote
  if (e != cudaSuccess) return cuda_fail("vsa_masked_attn_bwd: lists and sums", e);
  kv.splits = splits;
  kv.part = splits > 1 ? reinterpret_cast<float*>(ws + w.part) : nullptr;
  kv.clean_a = pa.clean_q;
  kv.clean_b = pa.clean_o;
  qq.clean_a = pa.clean_k;
  const bool cap = p.cap > 0.0f, bias = p.slopes != nullptr;
  if (cap) return bias ? launch<true, true>(kv, qq, m, stream) : launch<true, false>(kv, qq, m, stream);
  return bias ? launch<false, true>(kv, qq, m, stream) : launch<false, false>(kv, qq, m, stream);
}

}  // extern "C"

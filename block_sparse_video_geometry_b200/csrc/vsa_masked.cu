// Dense attention with capped scores, a distance bias, document and prefix
// masks: forward pass.
//
// Mathematics, per row: x_j = log2(e) * score_j, running maximum m and sum
// l = sum 2^(x_j - m), O = sum 2^(x_j - m) v_j; out = O / l, lse = ln2 (m + log2 l).
// Partial results over parts of the key axis join by their lse.
//
// Bound: tensor pipe (4 * 128 FLOP per visible pair) next to the exponentials (one
// per pair; a cap and a bias cost seven more FMA operations); one query over a long
// cache: HBM (k and v read once). Measured: 8192 x 8192, 24 heads 820 us (1010
// TFLOP/s; 938 us back to back under the power cap), one query over 4 x 33,001 keys
// 99-101 us (82% of the copy rate), 2 x 1,111 queries over 5,003 keys with cap and bias
// 205 us.
//
// Design. A block owns 256 rows of one head as two M = 128 tiles (slots) and walks
// the key tiles of 128. One warp copies K and V tiles (TMA) into a ring of five 32 KB
// stages; two warps issue the products, one for each slot; two groups of four warps,
// one for each slot too, run the softmax, a thread per row. Scores come in two
// buffers of 64 keys per query tile; P (bf16, the A operand of O += P V) overwrites
// its scores in TMEM, and the next scores follow behind that product. The softmax's
// reference is raised, and O rescaled in TMEM, only when a row's sum of P in a tile
// passes 2^32. Few rows: blocks of 128 rows, whose two slots take the key tiles in
// turn with the same queries and join their results in shared memory. Few queries (a
// new token over a cache): the heads that share a key head are packed into one tile,
// and the key axis is split over blocks; a second kernel joins the parts. Up to 128
// queries keep two bf16 terms of each P (see masked_fwd_kernel).
// Tiles that no row of the block sees are skipped: by arithmetic for causal
// masks, by a list that plan_kernel makes from the tiles' document ranges.
// Every wait is bounded (see vsa_masked_attn_status).

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "masked_scores.cuh"
#include "sm100.cuh"
#include "vsa_masked.h"

namespace vsa {
namespace masked {

using namespace sm100;

// ------------------------------------------------------------------- host
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

vsa_status encode(CUtensorMap* map, const void* data, int64_t S, int64_t heads, int64_t B, int64_t ss, int64_t sh,
                  int64_t sb) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return cuda_fail("cuTensorMapEncodeTiled is not available");
  const cuuint64_t dims[4] = {kHeadDim, static_cast<cuuint64_t>(S), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(ss) * 2, static_cast<cuuint64_t>(sh) * 2,
                                 static_cast<cuuint64_t>(sb) * 2};
  const cuuint32_t box[4] = {64, kRows, 1, 1}, one[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(data), dims, strides, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? VSA_OK : cuda_fail("cuTensorMapEncodeTiled refused a view");
}

}  // namespace

// A dimension of size 1 or stride 0 (broadcast) is given to the map with extent
// 1; the kernels use coordinate 0 for it.
vsa_status make_map(CUtensorMap* map, const vsa_view* v, int32_t B, int32_t S) {
  const Strides st = view_strides(v, B, S);
  return encode(map, v->data, S, st.h ? v->heads : 1, st.b ? B : 1, S > 1 ? st.s : kHeadDim, st.h ? st.h : kHeadDim,
                st.b ? st.b : kHeadDim);
}

vsa_status make_map(CUtensorMap* map, const uint16_t* copy, int32_t B, int32_t S, int32_t heads) {
  const int64_t row = static_cast<int64_t>(heads) * kHeadDim;
  return encode(map, copy, S, heads, B, row, kHeadDim, row * S);
}

vsa_status check(const vsa_mask* m, const vsa_mask_terms* t, int32_t B, int32_t Sq, int32_t Sk, int32_t Hq, int32_t Hk,
                 Problem* p) {
  if (!m || (m->mode != VSA_MASK_FULL && m->mode != VSA_MASK_CAUSAL)) return VSA_ERR_INVALID_ARG;
  if (m->documents != 0 && m->documents != 1) return VSA_ERR_INVALID_ARG;
  if (!std::isfinite(m->scale) || !std::isfinite(m->softcap) || m->softcap < 0.0f) return VSA_ERR_INVALID_ARG;
  if (B < 0 || Sq < 0 || Sk < 0 || Hq <= 0 || Hk <= 0 || Hq % Hk) return VSA_ERR_INVALID_ARG;
  if (B > 65535 || Hq > 65535 || Sq > kMaxPositions || Sk > kMaxPositions) return VSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * Hq * tiles(std::max(Sq, Sk)) > INT32_MAX / 32) return VSA_ERR_UNSUPPORTED;
  *p = Problem{};
  p->B = B;
  p->Hq = Hq;
  p->Hk = Hk;
  p->group = Hq / Hk;
  p->Sq = Sq;
  p->Sk = Sk;
  p->off = Sk - Sq;
  p->nkt = tiles(Sk);
  p->causal = m->mode == VSA_MASK_CAUSAL;
  p->documents = m->documents;
  p->masked = m->documents || (p->causal && Sq > 1);
  p->scale = m->scale > 0.0f ? m->scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(kHeadDim)));
  p->cap = m->softcap;
  if (!t) return m->documents ? VSA_ERR_INVALID_ARG : VSA_OK;
  const bool empty = B == 0 || Sq == 0 || Sk == 0;
  if (!empty && m->documents != (t->doc_q != nullptr)) return VSA_ERR_INVALID_ARG;
  if (!empty && m->documents != (t->doc_k != nullptr)) return VSA_ERR_INVALID_ARG;
  if (t->prefix && !p->causal) return VSA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(t->doc_q), static_cast<const void*>(t->doc_k),
                        static_cast<const void*>(t->prefix), static_cast<const void*>(t->slopes)})
    if (reinterpret_cast<uintptr_t>(x) % 4) return VSA_ERR_INVALID_ARG;
  if (m->documents && B > 1 && (t->doc_q_stride_b < 0 || t->doc_k_stride_b < 0)) return VSA_ERR_INVALID_ARG;
  p->doc_q = t->doc_q;
  p->doc_k = t->doc_k;
  p->doc_q_sb = B > 1 ? t->doc_q_stride_b : 0;
  p->doc_k_sb = B > 1 ? t->doc_k_stride_b : 0;
  p->prefix = t->prefix;
  p->slopes = t->slopes;
  return VSA_OK;
}

vsa_status check_tensor(const vsa_view* v, int32_t B, int32_t S, int32_t heads, bool output) {
  const vsa_status st = check_view(v, B, S, kHeadDim, 16, output);
  if (st != VSA_OK) return st;
  if (v->heads != heads || v->dtype != VSA_BF16) return VSA_ERR_INVALID_ARG;
  if (S > 1 && B > 0 && v->stride_s == 0) return VSA_ERR_UNSUPPORTED;
  // a tensor map's strides stay below 2^40 bytes
  const Strides s = view_strides(v, B, S);
  for (int64_t x : {s.b, s.s, s.h})
    if (x >= (int64_t{1} << 39)) return VSA_ERR_UNSUPPORTED;
  return VSA_OK;
}

// ------------------------------------------------------------- small kernels
namespace {

// Rows of v with an infinity or NaN, and the tiles' copies without them. One block
// per (head, tile) in x and batch entry, heads first: neighbours read neighbouring memory.
// HBM bound: v read once.
__global__ void __launch_bounds__(kTileThreads)
scan_kernel(const uint16_t* __restrict__ x, Strides st, int S, int heads, int n_tiles, Clean c) {
  const int h = blockIdx.x % heads, tile = blockIdx.x / heads, b = blockIdx.y;
  __shared__ uint32_t bad[4];
  if (threadIdx.x < 4) bad[threadIdx.x] = 0;
  uint4 w[kPieces];
  load_pieces(w, x + b * st.b + h * st.h + static_cast<int64_t>(tile) * kRows * st.s, st.s, min(kRows, S - tile * kRows));
  __syncthreads();
  find_bad(w, bad);
  __syncthreads();
  write_clean(c, w, bad, b, h, heads, tile, n_tiles, S);
}

// Smallest and largest document of positions [i0, i0 + n) of a row of ids
// (INT_MAX, -1 when all are padding) and whether one is padding; one warp.
struct Range {
  int lo, hi, pad;
};
__device__ __forceinline__ Range doc_range(const int32_t* ids, int i0, int n) {
  Range r{INT_MAX, -1, 0};
  for (int i = threadIdx.x & 31; i < n; i += 32) {
    const int d = ids[i0 + i];
    if (d >= 0) {
      r.lo = min(r.lo, d);
      r.hi = max(r.hi, d);
    } else {
      r.pad = 1;
    }
  }
  r.lo = __reduce_min_sync(0xffffffffu, r.lo);
  r.hi = __reduce_max_sync(0xffffffffu, r.hi);
  r.pad = __reduce_or_sync(0xffffffffu, r.pad);
  return r;
}

// Document ranges of the tiles of ids [B, S]: [B][tiles].
__global__ void __launch_bounds__(128)
range_kernel(const int32_t* __restrict__ ids, int64_t sb, int S, int n_tiles, int4* __restrict__ range) {
  const int tile = blockIdx.x * 4 + (threadIdx.x >> 5), b = blockIdx.y;
  if (tile >= n_tiles) return;
  const Range r = doc_range(ids + b * sb, tile * kRows, min(kRows, S - tile * kRows));
  if ((threadIdx.x & 31) == 0) range[static_cast<size_t>(b) * n_tiles + tile] = make_int4(r.lo, r.hi, r.pad, 0);
}

__device__ __forceinline__ bool meet(int4 a, int4 b) { return a.x <= b.y && b.x <= a.y; }
__device__ __forceinline__ bool one_doc(int4 a) { return a.x == a.y && !a.z; }
__device__ __forceinline__ bool same(int4 a, int4 b) { return one_doc(a) && one_doc(b) && a.x == b.x; }

// Appends the records (>= 0) of a block's 256 threads to `out` from `total`, in
// thread order; returns the new total.
__device__ __forceinline__ int append(int rec, int total, int32_t* out, int* n_warp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t vote = __ballot_sync(0xffffffffu, rec >= 0);
  if (lane == 0) n_warp[warp] = __popc(vote);
  __syncthreads();
  int at = total;
  for (int w = 0; w < 8; ++w) {
    at += w < warp ? n_warp[w] : 0;
    total += n_warp[w];
  }
  if (rec >= 0) out[at + __popc(vote & ((1u << lane) - 1u))] = rec;
  __syncthreads();
  return total;
}

// Key tiles that some row of a query block sees, ascending. One block per (query
// block, batch entry).
__global__ void __launch_bounds__(256)
plan_kernel(const __grid_constant__ Problem p, const int4* __restrict__ range, PlanRows rows, int n_blocks,
            int32_t* __restrict__ count, int32_t* __restrict__ list) {
  const int qb = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ int4 q[2];
  __shared__ int n_warp[8];
  if (warp < 2) {
    const int i0 = rows == kPlanAll ? 0 : rows == kPlanPairs ? (qb * 2 + warp) * kRows : qb * kRows;
    const int n = rows == kPlanAll ? p.Sq : max(0, min(kRows, p.Sq - i0));
    const Range r = doc_range(p.doc_q + b * p.doc_q_sb, min(i0, p.Sq), n);
    if (lane == 0) q[warp] = make_int4(r.lo, r.hi, r.pad, n > 0 ? p.limit(b, i0 + n - 1) : -1);
  }
  __syncthreads();
  int total = 0;
  int32_t* out = list + (static_cast<size_t>(b) * n_blocks + qb) * p.nkt;
  for (int t0 = 0; t0 < p.nkt; t0 += 256) {
    const int kt = t0 + threadIdx.x;
    int rec = -1;
    if (kt < p.nkt) {
      const int4 k = range[static_cast<size_t>(b) * p.nkt + kt];
      bool any = false;
      int flags = 0;
      for (int t = 0; t < 2; ++t) {
        any |= meet(k, q[t]) && kt * kRows <= q[t].w;
        if (!same(k, q[t])) flags |= t ? kPartial1 : kPartial0;
      }
      if (any) rec = kt | flags | (one_doc(k) ? kOneDoc : 0);
    }
    total = append(rec, total, out, n_warp);
  }
  if (threadIdx.x == 0) count[static_cast<size_t>(b) * n_blocks + qb] = total;
}

// Query tiles that see some key of a key tile, ascending. One block per (key
// tile, batch entry).
__global__ void __launch_bounds__(256)
plan_keys_kernel(const __grid_constant__ Problem p, const int4* __restrict__ range, const int4* __restrict__ range_q,
                 int nqt, int32_t* __restrict__ count, int32_t* __restrict__ list) {
  const int kt = blockIdx.x, b = blockIdx.y;
  __shared__ int n_warp[8];
  const int4 k = range[static_cast<size_t>(b) * p.nkt + kt];
  int total = 0;
  int32_t* out = list + (static_cast<size_t>(b) * p.nkt + kt) * nqt;
  for (int t0 = 0; t0 < nqt; t0 += 256) {
    const int qt = t0 + threadIdx.x;
    int rec = -1;
    if (qt < nqt) {
      const int4 q = range_q[static_cast<size_t>(b) * nqt + qt];
      if (meet(k, q) && kt * kRows <= p.limit(b, min((qt + 1) * kRows, p.Sq) - 1))
        rec = qt | (same(k, q) ? 0 : kPartial0) | (one_doc(q) ? kOneDoc : 0);
    }
    total = append(rec, total, out, n_warp);
  }
  if (threadIdx.x == 0) count[static_cast<size_t>(b) * p.nkt + kt] = total;
}

// --------------------------------------------------------------- main kernel
constexpr int kStages = 5;
constexpr int kThreads = 352;
constexpr int kWarpLoad = 8, kWarpMma = 9;          // warps 0-7: softmax; 9, 10: products of slot 0, 1
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;          // score buffer hb of slot t: 128 t + 64 hb; O of slot t: 256 + 128 t
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 64, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, 0, 1);
constexpr float kSumLimit = 4294967296.0f;          // 2^32: see the softmax step

struct Smem {
  uint8_t q[2][kTileBytes];
  uint8_t kv[kStages][kTileBytes];
  uint64_t full[2][kStages], empty[kStages];   // full: see count_of
  uint64_t q_full, s_full[2][2], p_full[2][2], pv_done[2], o_full[2], drain[2];   // [slot][score buffer]
  uint64_t joined;                   // one tile: both slots' halves of O, maxima and sums are in shared memory
  float m[2][kRows], l[2][kRows];
  uint32_t tmem_base;
  int abort;
};

struct Args {
  Problem p;
  const uint16_t* q;
  Strides sq;
  int32_t k_h, k_b, v_h, v_b;        // 1: the map has that dimension, 0: broadcast
  Clean clean_v;                     // bad == null: v is not scanned
  uint16_t* out;
  Strides so;
  float* lse;
  const int32_t* count;              // plan of visible tiles, or null
  const int32_t* list;
  int32_t packed;                    // rows = (head of the group, query), unit = key head; else unit = query head
  int32_t units, rows, n_blocks;     // rows of a unit, blocks of them
  int32_t one_tile;                  // blocks of 128 rows, which both slots hold, taking turns over the key tiles; else 256
  int32_t splits;                    // parts of the key axis
  float* part_o;                     // [split][B][Hq][Sq][128], or null (splits == 1)
  float* part_lse;                   // [split][B][Hq][Sq], log2
  int* err;
};

__device__ __forceinline__ bool bounded_wait(Smem& sm, uint64_t& bar, uint32_t parity, int* err) {
  bool ok = mbar_wait(smem_u32(&bar), parity, &sm.abort, kTimeoutNs);
  if (!ok) {
    *reinterpret_cast<volatile int*>(err) = VSA_ERR_TIMEOUT;
    *reinterpret_cast<volatile int*>(&sm.abort) = 1;
  }
  return ok;
}
// Every lane waits; the warp leaves together.
__device__ __forceinline__ bool warp_wait(Smem& sm, uint64_t& bar, uint32_t parity, int* err) {
  return __all_sync(0xffffffffu, bounded_wait(sm, bar, parity, err));
}

// What the bf16 pair `first` left of p0 and p1, as bf16 again.
__device__ __forceinline__ uint32_t second_term(uint32_t first, float p0, float p1) {
  const uint64_t f = pack_f32x2(__uint_as_float(first << 16), __uint_as_float(first & 0xFFFF0000u));
  unpack_f32x2(fma_f32x2(f, pack_f32x2(-1.0f, -1.0f), pack_f32x2(p0, p1)), p0, p1);
  return pack_bf16x2(p0, p1);
}

// kFine: P enters the second product as two bf16 terms, its rounding and what that left
// (2^-16 of it together), so that the output is off by its own rounding only. One term
// makes a long sum's relative error 0.0023-0.0026 instead of 0.0017. Taken for up to 128
// queries, whose blocks wait for HBM: one query over 4 x 33,001 keys 95.7 us with one
// term, 98.6 with two (with cap and bias 120 and 132); 128 queries over 8,000 keys, 4 x 48
// heads 181 and 189. Longer calls would pay 2 to 22% (8192 x 24 heads 830 -> 1014 us).
template <bool kCap, bool kBias, bool kFine>
__global__ void __launch_bounds__(kThreads, 1)
masked_fwd_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_vc) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {          // swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicExch(a.err, VSA_ERR_UNSUPPORTED);
    return;
  }
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  const Problem& p = a.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool one = kFine || a.one_tile;

  // block -> (query block, split, unit, batch entry); late query blocks, the
  // longest under a causal mask, first
  int id = blockIdx.x;
  const int per = a.units * p.B * a.splits;
  const int qb = a.n_blocks - 1 - id / per;
  id %= per;
  const int split = id % a.splits;
  id /= a.splits;
  const int unit = id % a.units, b = id / a.units;
  const int hk = a.packed ? unit : unit / p.group;

  // key tiles of this block: entries [s0, s1) of its list (or the numbers themselves)
  const size_t plan_row = static_cast<size_t>(b) * a.n_blocks + qb;
  int n_all;
  if (a.count) {
    n_all = a.count[plan_row];
  } else {
    const int last = a.packed ? p.Sq - 1 : min((qb + 1) * (one ? kRows : 2 * kRows), p.Sq) - 1;
    n_all = max(0, p.limit(b, last) + kRows) / kRows;     // tiles up to the last row's limit (none: below 0)
  }

  if (threadIdx.x == 32 * kWarpLoad) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sm.full[0][i]), 1);
      mbar_init(smem_u32(&sm.full[1][i]), 1);
      mbar_init(smem_u32(&sm.empty[i]), one ? 1 : 2);     // a stage is read by one slot, or by both
    }
    mbar_init(smem_u32(&sm.q_full), 8);
    mbar_init(smem_u32(&sm.joined), 8);
    for (int t = 0; t < 2; ++t) {
      for (int hb = 0; hb < 2; ++hb) {
        mbar_init(smem_u32(&sm.s_full[t][hb]), 1);
        mbar_init(smem_u32(&sm.p_full[t][hb]), 4);
      }
      mbar_init(smem_u32(&sm.pv_done[t]), 1);
      mbar_init(smem_u32(&sm.o_full[t]), 1);
      mbar_init(smem_u32(&sm.drain[t]), 1);
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(smem_u32(&sm.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (warp < 8) {
    // rows of Q into shared memory, 16 lanes per row (rows past the end: zero), all
    // loads in flight at once; one tile: both slots' threads (one by one, behind the
    // block's first barrier, its first product waited 6-10 us)
    const int t = warp >> 2, r = threadIdx.x & 127;
    const int rows0 = one ? qb * kRows + 64 * t : (2 * qb + t) * kRows;   // this slot's share
    const int n_it = one ? 8 : 16;
    uint4 w[16];
#pragma unroll
    for (int it = 0; it < 16; ++it) {
      const int e = it * 128 + r, c = e & 15, at = rows0 + (e >> 4);
      w[it] = make_uint4(0, 0, 0, 0);
      if (it < n_it && at < a.rows) {
        const int gg = a.packed ? at / p.Sq : 0, i = a.packed ? at - gg * p.Sq : at;
        const int hh = a.packed ? hk * p.group + gg : unit;
        w[it] = *reinterpret_cast<const uint4*>(a.q + b * a.sq.b + i * a.sq.s + hh * a.sq.h + c * 8);
      }
    }
#pragma unroll
    for (int it = 0; it < 16; ++it) {
      const int e = it * 128 + r, c = e & 15, rr = (one ? 64 * t : 0) + (e >> 4);
      if (it < n_it)
        *reinterpret_cast<uint4*>(sm.q[one ? 0 : t] + (c >> 3) * 16384 + rr * 128 + ((c & 7) ^ (rr & 7)) * 16) = w[it];
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  const int32_t* list = a.count ? a.list + plan_row * p.nkt : nullptr;
  const int s0 = static_cast<int>(static_cast<int64_t>(n_all) * split / a.splits);
  const int s1 = static_cast<int>(static_cast<int64_t>(n_all) * (split + 1) / a.splits);
  // last tile first: under a distance bias the largest scores are near the
  // query, and a reference found there rarely has to be raised
  const int n = s1 - s0;
  const uint4* bad = a.clean_v.bad ? a.clean_v.bad + (static_cast<size_t>(b) * p.Hk + hk) * p.nkt : nullptr;

  // Place of K or V of key tile j in loading order; place % kStages is its stage. With
  // one tile the slots hold two key tiles' scores at a time, so K runs two tiles ahead
  // of V.
  const int ahead = one ? 2 : 1;
  auto place_k = [&](int j) { return j + max(0, j - ahead + 1); };
  auto place_v = [&](int j) { return j + min(n, j + ahead); };
  // Count of the barrier that its landing completes, full[one ? j & 1 : 0][count %
  // kStages]. A barrier's parity tells its phases apart only for one who saw the
  // last. Both slots see every stage of two tiles; with one tile each sees its own key
  // tiles only, so that the slots have barriers of their own, counted over their own
  // stages (K and V in turn). A count comes round, kStages of them later, behind at
  // least kStages stages of the ring: the stage before has been read, and seen, by then.
  auto count_of = [&](int j, bool v) { return one ? (j & ~1) + v : v ? place_v(j) : place_k(j); };

  if (warp == kWarpLoad) {
    if (lane == 0) {
      prefetch_map(&map_k);
      prefetch_map(&map_v);
      bool ok = true;
      int e = 0, kj = 0, vj = 0;
      for (; e < 2 * n; ++e) {
        // the order in which the products use them: K up to `ahead` tiles before V
        const bool is_v = kj == min(n, vj + ahead);
        const int st = e % kStages, j = is_v ? vj++ : kj++;
        const int kt = (list ? list[s1 - 1 - j] : s1 - 1 - j) & kTileMask;
        if (e >= kStages && !(ok = bounded_wait(sm, sm.empty[st], (e / kStages - 1) & 1, a.err))) break;
        const CUtensorMap* map = is_v ? &map_v : &map_k;
        int h = (is_v ? a.v_h : a.k_h) ? hk : 0, bb = (is_v ? a.v_b : a.k_b) ? b : 0;
        if (is_v && bad) {
          const uint4 m = bad[kt];
          if (m.x | m.y | m.z | m.w) map = &map_vc, h = hk, bb = b;
        }
        const uint32_t bar = smem_u32(&sm.full[one ? j & 1 : 0][count_of(j, is_v) % kStages]), dst = smem_u32(sm.kv[st]);
        mbar_arrive_expect_tx(bar, kTileBytes);
        tma_load_4d(dst, map, 0, kt * kRows, h, bb, bar);
        tma_load_4d(dst + kTileBytes / 2, map, 64, kt * kRows, h, bb, bar);
      }
      if (!ok) {                                           // every issued copy lands before the block exits
        kj = vj = 0;
        for (int i = 0; i < e; ++i) {
          const bool is_v = kj == min(n, vj + ahead);
          const int j = is_v ? vj++ : kj++, c = count_of(j, is_v);
          if (i >= e - kStages)
            mbar_wait(smem_u32(&sm.full[one ? j & 1 : 0][c % kStages]), (c / kStages) & 1, nullptr, kDrainNs);
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma || warp == kWarpMma + 1) {
    // One issuing warp per slot: while one waits, the other's products run. (One
    // warp for both lost the 100 cycles of every wait to the tensor pipe: 1214 us
    // instead of 868 for 8192 x 24 heads.) Each slot has two score buffers of 64
    // keys, so that the next scores are there when its softmax ends one buffer;
    // with one buffer of 128 keys the chain S, softmax, P V of a slot bounded a step
    // (910 us).
    const int t = warp - kWarpMma;
    const uint32_t ts = tmem + kColS + 128 * t, to = tmem + kColO + 128 * t;
    const uint64_t qd = smem_desc_sw128(smem_u32(sm.q[one ? 0 : t]), 16, 1024);
    bool ok = warp_wait(sm, sm.q_full, 0, a.err);
    auto landed = [&](int j, bool v) {
      const int c = count_of(j, v);
      return warp_wait(sm, sm.full[one ? t : 0][c % kStages], (c / kStages) & 1, a.err);
    };
    // S(j, hb) = Q K^T over half hb of key tile j: 16 channels per K step, 32 B
    // inside a swizzled row of the d half kk / 4; 64 key rows = 8 KB.
    auto scores = [&](int j, int hb) {
      const int st = place_k(j) % kStages;
      if (hb == 0 && !landed(j, false)) return false;
      tc_fence_after();
      const uint64_t kd = smem_desc_sw128(smem_u32(sm.kv[st]) + 8192 * hb, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ss(ts + 64 * hb, qd + (kk >> 2) * (16384 >> 4) + (kk & 3) * 2,
                  kd + (kk >> 2) * (16384 >> 4) + (kk & 3) * 2, kIdescS, kk > 0 ? 1u : 0u);
        umma_commit(smem_u32(&sm.s_full[t][hb]));
        if (hb == 1) umma_commit(smem_u32(&sm.empty[st]));
      }
      __syncwarp();
      return true;
    };
    const int step = one ? 2 : 1, j0 = one ? t : 0;
    if (ok && j0 < n) ok = scores(j0, 0) && scores(j0, 1);
    for (int j = j0, i = 0; ok && j < n; j += step, ++i) {
      const int st = place_v(j) % kStages;
      if (!(ok = landed(j, true))) break;
#pragma unroll 1
      for (int hb = 0; hb < 2; ++hb) {
        if (!(ok = warp_wait(sm, sm.p_full[t][hb], i & 1, a.err))) break;
        tc_fence_after();
        // V as MN-major B: d halves 16 KB apart, 16 keys = 2 KB per K step; P (A,
        // over its scores): 16 keys = 8 columns of bf16 pairs
        const uint64_t vd = smem_desc_sw128(smem_u32(sm.kv[st]) + 8192 * hb, 16384, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            // two terms: the first of 32 keys over 16 of their columns, the second over the others
            const uint32_t p = ts + 64 * hb + (kFine ? (kk >> 1) * 32 + (kk & 1) * 8 : kk * 8);
            umma_ts(to, p, vd + kk * (2048 >> 4), kIdescPV, i > 0 || hb > 0 || kk > 0 ? 1u : 0u);
            if constexpr (kFine) umma_ts(to, p + 16, vd + kk * (2048 >> 4), kIdescPV, 1u);
          }
          umma_commit(smem_u32(&sm.pv_done[t]));
          if (hb == 1) umma_commit(smem_u32(&sm.empty[st]));
          if (hb == 1 && j + step >= n) umma_commit(smem_u32(&sm.o_full[t]));
        }
        __syncwarp();
        if (j + step < n && !(ok = scores(j + step, hb))) break;
      }
    }
    if (!ok && elect_one()) {
      umma_commit(smem_u32(&sm.drain[t]));
      mbar_wait(smem_u32(&sm.drain[t]), 0, nullptr, kDrainNs);
    }
    __syncwarp();
  } else if (warp < 8) {
    const int t = warp >> 2;                               // tile (or slot)
    const int r = threadIdx.x & 127;                       // row of the tile = TMEM lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t ts = lane_addr + kColS + 128 * t, to = lane_addr + kColO + 128 * t;
    const int tile_row0 = one ? qb * kRows : (2 * qb + t) * kRows;
    const int row = tile_row0 + r;
    const bool live = row < a.rows;
    const int g = a.packed ? row / p.Sq : 0;
    const int i_q = min(a.packed ? row - g * p.Sq : row, p.Sq - 1);
    const int h = a.packed ? min(hk * p.group + g, p.Hq - 1) : unit;
    const int lim = kFine && !live ? -1 : p.limit(b, i_q);   // few queries: warps without any row skip the softmax
    // smallest limit of the tile's rows: tiles up to there are seen by all of them
    const int lim0 = p.limit(b, a.packed ? 0 : min(tile_row0, p.Sq - 1));
    const int doc = p.documents && live ? p.doc_q[b * p.doc_q_sb + i_q] : -1;
    const int32_t* dk = p.documents ? p.doc_k + b * p.doc_k_sb : nullptr;
    const ScoreTerms terms(p.scale, p.cap, kBias ? p.slopes[h] : 0.0f);
    if (lane == 0) mbar_arrive(smem_u32(&sm.q_full));

    float m = -INFINITY, l = 0.0f;
    bool ok = true, fresh = true;              // fresh: no half tile so far had a row that sees some of it
    const int step = one ? 2 : 1;
    int i = 0;
    for (int j = one ? t : 0; j < n; j += step, ++i) {
      const int rec = list ? list[s1 - 1 - j] : s1 - 1 - j;
      const int kt = rec & kTileMask, k0 = kt * kRows;
      // a tile of one document is hidden from a row as a whole or not at all
      const bool by_doc = rec & (t ? kPartial1 : kPartial0), part_doc = by_doc && !(rec & kOneDoc);
      const bool partial = by_doc || k0 + kRows - 1 > lim0;
      const int lim_t = by_doc && !part_doc && (doc < 0 || __ldg(dk + k0) != doc) ? -1 : lim;
      uint4 bm = make_uint4(0, 0, 0, 0);
      if (bad) bm = bad[kt];
      const bool flagged = bm.x | bm.y | bm.z | bm.w;
      for (int hb = 0; hb < 2; ++hb) {
        const uint32_t tb = ts + 64 * hb;                    // this half's scores
        if (!(ok = warp_wait(sm, sm.s_full[t][hb], i & 1, a.err))) break;
        tc_fence_after();
        // A row that sees none of the half by order or by the tile's document waits for
        // its reference; a warp of such rows has P = 0. (Blocks across two documents had
        // their second rows' references sought at every tile of the first: 146 us
        // for 40 tiles, so 96.)
        const bool none = lim_t < k0 + 64 * hb;
        if (__all_sync(0xffffffffu, none)) {
          uint32_t zero[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) zero[u] = 0;
          for (int q2 = 0; q2 < (kFine ? 4 : 2); ++q2) tmem_st32x16(tb + 16 * q2, zero);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[t][hb]));
          continue;
        }
        // scores of key columns [32 q4, 32 q4 + 32) in place -> log2 units minus a
        // reference: cap, bias, mask
        auto finish = [&](int q4, float (&x)[32], float minus_ref) {
          const int col = 32 * q4;
          float tanhs[32];
          score_args<kCap, kBias>(x, tanhs, terms, static_cast<float>(i_q + p.off - k0 - col), -1.0f,
                                  [&](int) { return pack_f32x2(minus_ref, minus_ref); });
          if (partial) {
            const int lc = lim_t - k0 - col;
#pragma unroll
            for (int u = 0; u < 32; ++u) x[u] = u <= lc ? x[u] : -INFINITY;
            if (part_doc) {
              const bool seeing = doc >= 0;
#pragma unroll
              for (int u = 0; u < 32; ++u) {
                const int d = __ldg(dk + min(k0 + col + u, p.Sk - 1));
                x[u] = seeing && d == doc ? x[u] : -INFINITY;
              }
            }
          }
          if (flagged) {
            // a visible key whose v holds an infinity or NaN makes the row NaN (its v is zero in the copy)
            const uint32_t bits = q4 == 0 ? bm.x : q4 == 1 ? bm.y : q4 == 2 ? bm.z : bm.w;
#pragma unroll
            for (int u = 0; u < 32; ++u)
              if (((bits >> u) & 1u) && x[u] != -INFINITY) x[u] = NAN;
          }
        };
        // P (bf16 pairs) against the reference m, and its 32-bit sum. Where no column
        // needs more than the pairwise form, each pair's arguments stand next to its
        // exponentials, so that the FMA pipe and the exponential unit run together.
        // A quarter of the exponentials go to the FMA pipe: 868 -> 834 us for 8192 x
        // 24 heads (an eighth 848, three eighths 862); none where the cap fills it.
        uint32_t w[2][16], w2[kFine ? 2 : 1][16];
        const float d0 = static_cast<float>(i_q + p.off - k0 - 64 * hb);
        float k_bias;
        const bool plain = one_side<kBias>(terms, d0, -1.0f, 64.0f, k_bias) && !partial && !flagged;
        auto exponentials = [&]() {
          const float ms = m == -INFINITY ? 0.0f : m;
          uint64_t ls[2] = {0, 0};
          float x[2][32];
          tmem_ld32x32f(tb, x[0]);
          tmem_wait_ld32(x[0]);
          tmem_ld32x32f(tb + 32, x[1]);
          auto take = [&](int q2, int u) {
            float p0 = x[q2][2 * u], p1 = x[q2][2 * u + 1];
            ex2_pair(p0, p1, !kCap && u % 4 == 2);
            ls[u & 1] = add_f32x2(ls[u & 1], pack_f32x2(p0, p1));
            w[q2][u] = pack_bf16x2(p0, p1);
            if constexpr (kFine) w2[q2][u] = second_term(w[q2][u], p0, p1);
          };
          bool pairwise = plain;
          if constexpr (kCap) {
            const float top = largest<kCap>(x[0]);
            tmem_wait_ld32(x[1]);
            pairwise = __all_sync(0xffffffffu, largest<kCap>(x[1], top) <= terms.limit) && plain;
          }
          if ((kCap || kBias) && pairwise) {
            const PairArgs<kCap, kBias> pair(terms, k_bias, d0, -1.0f, -ms);
#pragma unroll
            for (int q2 = 0; q2 < 2; ++q2) {
              if (q2 && !kCap) tmem_wait_ld32(x[1]);
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                uint64_t q;
                unpack_f32x2(pair(pack_f32x2(x[q2][2 * u], x[q2][2 * u + 1]), 32 * q2 + 2 * u, q), x[q2][2 * u],
                             x[q2][2 * u + 1]);
                take(q2, u);
              }
            }
          } else {
#pragma unroll
            for (int q2 = 0; q2 < 2; ++q2) {
              if (q2 && !kCap) tmem_wait_ld32(x[1]);
              finish(2 * hb + q2, x[q2], -ms);
#pragma unroll
              for (int u = 0; u < 16; ++u) take(q2, u);
            }
          }
          float s0, s1;
          unpack_f32x2(add_f32x2(ls[0], ls[1]), s0, s1);
          return s0 + s1;
        };
        // The reference m is a maximum of some earlier half tile. P, its sums and O
        // are floats of the 32-bit range (bf16 has it too), so a reference that is
        // too low costs no precision; while a row's sum of P stays within 2^32,
        // neither a maximum nor a rescale of O is needed. Otherwise (and on the
        // first visible key) the exact maximum is formed, O (complete up to the
        // last half) and l are rescaled and P is formed again.
        auto rise = [&](bool raise) {
          float top = -INFINITY;
#pragma unroll 1
          for (int q2 = 0; q2 < 2; ++q2) {
            float x[32];
            tmem_ld32x32f(tb + 32 * q2, x);
            tmem_wait_ld32(x);
            finish(2 * hb + q2, x, 0.0f);
#pragma unroll
            for (int u = 0; u < 32; ++u) top = fmaxf(top, x[u]);
          }
          const bool grow = raise && top > m;
          const float f = grow ? ex2_approx(m - top) : 1.0f;   // m = -inf: 0, and l and O are 0
          if (grow) m = top;
          l *= f;
          const int halves = 2 * i + hb;                       // P V products so far
          if (halves > 0) {
            if (!(ok = warp_wait(sm, sm.pv_done[t], (halves - 1) & 1, a.err))) return;
            tc_fence_after();
#pragma unroll 1
            for (int q4 = 0; q4 < 4; ++q4) {
              float o[32];
              tmem_ld32x32f(to + 32 * q4, o);
              tmem_wait_ld32(o);
              uint32_t ow[32];
#pragma unroll
              for (int u = 0; u < 32; ++u) ow[u] = __float_as_uint(o[u] * f);
              tmem_st32x32(to + 32 * q4, ow);
            }
          }
        };
        // The first half tile that a row of the warp sees: the scores are finished once, back into
        // their columns, and their exact maximum is the reference. (O and l are zero, or
        // NaN, so nothing is rescaled.) Without cap and bias, whose scores are quickly
        // finished twice, the form costs more in the main loop than it saves (dense 8192
        // x 24 heads 833 -> 858 us).
        auto begin = [&]() {
          float top = -INFINITY;
#pragma unroll 1
          for (int q2 = 0; q2 < 2; ++q2) {
            float x[32];
            uint32_t y[32];
            tmem_ld32x32f(tb + 32 * q2, x);
            tmem_wait_ld32(x);
            finish(2 * hb + q2, x, 0.0f);
#pragma unroll
            for (int u = 0; u < 32; ++u) {
              top = fmaxf(top, x[u]);
              y[u] = __float_as_uint(x[u]);
            }
            tmem_st32x32(tb + 32 * q2, y);
          }
          tmem_wait_st();
          m = fmaxf(m, top);
          const float ms = m == -INFINITY ? 0.0f : m;
          uint64_t sum = 0;
          const uint64_t minus = pack_f32x2(-ms, -ms);
#pragma unroll 1
          for (int q2 = 0; q2 < 2; ++q2) {                     // P of 32 columns ends up over scores already read
            float x[32];
            uint32_t y[16], y2[16];
            tmem_ld32x32f(tb + 32 * q2, x);
            tmem_wait_ld32(x);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              float p0, p1;
              unpack_f32x2(add_f32x2(pack_f32x2(x[2 * u], x[2 * u + 1]), minus), p0, p1);
              ex2_pair(p0, p1, false);
              sum = add_f32x2(sum, pack_f32x2(p0, p1));
              y[u] = pack_bf16x2(p0, p1);
              if constexpr (kFine) y2[u] = second_term(y[u], p0, p1);
            }
            tmem_st32x16(tb + (kFine ? 32 : 16) * q2, y);
            if constexpr (kFine) tmem_st32x16(tb + 32 * q2 + 16, y2);
          }
          float s0, s1;
          unpack_f32x2(sum, s0, s1);
          return s0 + s1;
        };
        float psum = INFINITY;
        // With cap or bias a row's bits depend on which of the forms it takes: that goes by
        // order and documents alone (`fresh`), not by whether another row of the warp has met
        // nothing but NaN, in a key that this row may not see.
        const bool first = kCap || kBias ? fresh : __all_sync(0xffffffffu, m == -INFINITY);
        const bool begun = (kCap || kBias) && first;
        fresh = false;
        if (begun) {
          psum = begin();
        } else if constexpr (kCap) {
          // one copy of the long capped exponentials in a loop (1,555 causal tokens 73 us
          // with two, 67 so; without a cap two copies are faster)
          bool raised = false, raise = false;
#pragma unroll 1
          for (;;) {
            if (raised) rise(raise);
            if (!ok) break;
            psum = exponentials();
            if (raised) break;
            raise = (m == -INFINITY && !none) || !(psum <= kSumLimit);   // the others of the warp keep theirs
            raised = __any_sync(0xffffffffu, raise);
            if (!raised) break;
          }
        } else {
          if (kBias || !first) psum = exponentials();
          const bool raise = (m == -INFINITY && !none) || !(psum <= kSumLimit);
          if (__any_sync(0xffffffffu, raise)) {
            rise(raise);
            if (ok) psum = exponentials();
          }
        }
        if (!ok) break;
        if (!begun) {
#pragma unroll
          for (int q2 = 0; q2 < 2; ++q2) {
            tmem_st32x16(tb + (kFine ? 32 : 16) * q2, w[q2]);
            if constexpr (kFine) tmem_st32x16(tb + 32 * q2 + 16, w2[q2]);
          }
        }
        l += psum;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[t][hb]));
      }
      if (!ok) break;
    }
    // ---------------------------------------------------------- epilogue
    if (ok && i > 0) {
      ok = warp_wait(sm, sm.o_full[t], 0, a.err);
      tc_fence_after();
    }
    // One tile: each slot joins its own 64 channels with the other's, which lie over Q,
    // [channel][row] (slot 0 joining all: 1 us a block more).
    float* held = reinterpret_cast<float*>(sm.q[0]);        // 64 KB over both Q tiles
    const int c0 = one ? 64 * t : 0, c1 = one ? c0 + 64 : kHeadDim;
    const bool other = one && n > 1;                        // both slots had a key tile
    float f0 = 1.0f, f1 = 0.0f;
    if (other && ok) {
      ok = warp_wait(sm, sm.o_full[t ^ 1], 0, a.err);       // its products read Q no longer
      if (ok) {
        sm.m[t][r] = m;
        sm.l[t][r] = l;
#pragma unroll 1
        for (int c = 64 - c0; c < 128 - c0; c += 32) {
          float o[32];
          tmem_ld32x32f(to + c, o);
          tmem_wait_ld32(o);
#pragma unroll
          for (int u = 0; u < 32; ++u) held[(c + u) * kRows + r] = o[u];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.joined));
        ok = warp_wait(sm, sm.joined, 0, a.err);
        const float mo = sm.m[t ^ 1][r], top = fmaxf(m, mo), ref = top == -INFINITY ? 0.0f : top;
        f0 = ex2_approx(m - ref);
        f1 = ex2_approx(mo - ref);
        l = l * f0 + sm.l[t ^ 1][r] * f1;
        m = top;
      }
    }
    if (ok && !(one && t == 1 && !other)) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const float lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
      const size_t at = (static_cast<size_t>(b) * p.Hq + h) * p.Sq + i_q;
      const size_t all = static_cast<size_t>(p.B) * p.Hq * p.Sq;
      if (live && !(one && t == 1)) {
        if (a.part_o) a.part_lse[split * all + at] = lse2;
        else a.lse[at] = lse2 * 0.6931471805599453f;
      }
      // bf16 rows of the output go through shared memory that no product reads any more
      // (Q, or where both slots' products have ended a stage of the ring), each warp's own
      // rows, so that whole rows are stored and not 16 bytes of 32 rows at a time.
      const int chunks = other ? 8 : 16;                    // 16-byte pieces of a row
      uint8_t* rows = (other ? sm.kv[t] : sm.q[t]) + (warp & 3) * 32 * chunks * 16;
#pragma unroll 1
      for (int c = c0; c < (other ? c1 : kHeadDim); c += 32) {
        float o[32];
        __syncwarp();
        if (i > 0) {
          tmem_ld32x32f(to + c, o);
          tmem_wait_ld32(o);
        } else {
#pragma unroll
          for (int u = 0; u < 32; ++u) o[u] = 0.0f;
        }
        if (other) {
#pragma unroll
          for (int u = 0; u < 32; ++u) o[u] = fmaf(held[(c + u) * kRows + r], f1, o[u] * f0);
        }
#pragma unroll
        for (int u = 0; u < 32; ++u) o[u] = l == 0.0f ? 0.0f : o[u] * inv;
        if (!a.part_o) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(rows + (lane * chunks + (((c - c0) / 8 + u) ^ (lane & (chunks - 1)))) * 16) =
                make_uint4(pack_bf16x2(o[8 * u], o[8 * u + 1]), pack_bf16x2(o[8 * u + 2], o[8 * u + 3]),
                           pack_bf16x2(o[8 * u + 4], o[8 * u + 5]), pack_bf16x2(o[8 * u + 6], o[8 * u + 7]));
        } else if (live) {
          float4* dst = reinterpret_cast<float4*>(a.part_o + (split * all + at) * kHeadDim + c);
#pragma unroll
          for (int u = 0; u < 8; ++u) dst[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
        }
      }
      if (!a.part_o) {
        const int64_t mine = live ? b * a.so.b + i_q * a.so.s + h * a.so.h : -1;   // the row's place in out
        __syncwarp();
        for (int it = 0; it < chunks; ++it) {
          const int e = it * 32 + lane, rr = e / chunks, k = e & (chunks - 1);
          const int64_t place = __shfl_sync(0xffffffffu, mine, rr);
          if (place >= 0)
            *reinterpret_cast<uint4*>(a.out + place + c0 + 8 * k) =
                *reinterpret_cast<const uint4*>(rows + (rr * chunks + (k ^ (rr & (chunks - 1)))) * 16);
        }
      }
    }
    tc_fence_before();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// out and lse from the parts over the key axis: one warp per row.
__global__ void __launch_bounds__(256)
join_kernel(const __grid_constant__ Args a) {
  const size_t all = static_cast<size_t>(a.p.B) * a.p.Hq * a.p.Sq;
  const size_t at = static_cast<size_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= all) return;
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  bool nan = false;
  for (int s = lane; s < a.splits; s += 32) {
    const float x = a.part_lse[s * all + at];
    top = fmaxf(top, x);
    nan |= isnan(x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (__any_sync(0xffffffffu, nan)) top = NAN;
  const float ref = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s = 0; s < a.splits; ++s) {
    const float w = exp2f(a.part_lse[s * all + at] - ref);
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + (s * all + at) * kHeadDim + lane * 4);
    sum += w;
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int i = static_cast<int>(at % a.p.Sq);
  const size_t bh = at / a.p.Sq;
  const int h = static_cast<int>(bh % a.p.Hq);
  const int64_t b = static_cast<int64_t>(bh / a.p.Hq);
  *reinterpret_cast<uint2*>(a.out + b * a.so.b + i * a.so.s + h * a.so.h + lane * 4) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (lane == 0) a.lse[at] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

// out = 0 and lse = -inf of every row (no keys).
__global__ void __launch_bounds__(256) empty_kernel(const __grid_constant__ Args a) {
  const size_t all = static_cast<size_t>(a.p.B) * a.p.Hq * a.p.Sq;
  const size_t at = static_cast<size_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= all) return;
  const int lane = threadIdx.x & 31;
  const int i = static_cast<int>(at % a.p.Sq);
  const size_t bh = at / a.p.Sq;
  const int h = static_cast<int>(bh % a.p.Hq);
  const int64_t b = static_cast<int64_t>(bh / a.p.Hq);
  *reinterpret_cast<uint2*>(a.out + b * a.so.b + i * a.so.s + h * a.so.h + lane * 4) = make_uint2(0u, 0u);
  if (lane == 0) a.lse[at] = -INFINITY;
}

// How the rows are laid over blocks, and how often the key axis is split.
struct Layout {
  int32_t packed, units, rows, n_blocks, one_tile, splits;
};

// The heads of a group share a tile when all their queries fit 128 rows. Blocks
// of 256 rows read each key tile once for two query tiles; blocks of 128 rows
// leave less of the GPU idle where blocks are few or of different length (2 x
// 1,111 queries over 5,003 keys, 24 heads: 240 or 432 blocks on 148 SMs). The key
// axis is split where there are fewer blocks than SMs. The choice is the least of an
// estimate in quarters of a 256-row block's key tile: for equal blocks the rounds
// they take, under a causal mask the work spread over all SMs and a third of the
// longest block; a block adds its start and end, splitting the joining pass.
Layout layout_of(const Problem& p) {
  Layout best{};
  best.packed = p.group > 1 && static_cast<int64_t>(p.group) * p.Sq <= kRows;
  best.units = best.packed ? p.Hk : p.Hq;
  best.rows = best.packed ? p.group * p.Sq : p.Sq;
  const double sms = device_sms(), pairs = static_cast<double>(best.units) * p.B;
  double least = 1e300;
  for (int one = best.rows <= kRows ? 1 : 0; one < 2; ++one) {
    const int per = one ? kRows : 2 * kRows, n_blocks = (best.rows + per - 1) / per;
    // one tile reads the key tile for half the rows; where no other block reads it, HBM bounds it
    const double tile = !one ? 4.0 : n_blocks > 1 ? 2.2 : 3.3, fixed = one && n_blocks == 1 ? 16.0 : 6.0;
    // key tiles of the blocks together, and of the longest
    double total = static_cast<double>(n_blocks) * p.nkt;
    bool unequal = p.causal && !best.packed && n_blocks > 1;
    if (unequal) {
      total = 0.0;
      for (int qb = 0; qb < n_blocks; ++qb)
        total += std::max(0, std::min(p.nkt, (std::min((qb + 1) * per, p.Sq) + p.off + kRows - 1) / kRows));
      // queries behind a long cache: as good as equal (300 over 20,000 keys, 8 heads: 144 blocks 79 us, 192 98 us)
      if (total > 0.95 * n_blocks * p.nkt) unequal = false;
    }
    for (int s = 1; s <= 64 && s <= std::max(1, p.nkt / 2); ++s) {
      const double longest = tile * ((p.nkt + s - 1) / s) + fixed, blocks = n_blocks * pairs * s;
      const double work = pairs * (tile * total + fixed * n_blocks * s) / sms;
      double t = unequal ? std::max(longest, work + longest / 3.0) : std::ceil(blocks / sms) * longest;
      // a split writes and reads its rows in 32 bits (0.45 us a unit, 6.5 TB/s) behind one more launch
      if (s > 1) t += 12.0 + pairs * best.rows * s * 1024.0 / 6.5e12 / 0.45e-6;
      if (t < least * 0.97) {
        least = t;
        best.n_blocks = n_blocks;
        best.one_tile = one;
        best.splits = s;
      }
    }
  }
  return best;
}

struct Workspace {
  size_t range, count, list, bad, copy, part_o, part_lse, total;
};

Workspace workspace_of(const Problem& p, const Layout& L) {
  Workspace w{};
  size_t off = kHeader;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  const size_t b = static_cast<size_t>(p.B), nkt = static_cast<size_t>(p.nkt), nb = static_cast<size_t>(L.n_blocks);
  if (p.documents) {
    w.range = take(b * nkt * sizeof(int4));
    w.count = take(b * nb * sizeof(int32_t));
    w.list = take(b * nb * nkt * sizeof(int32_t));
  }
  if (p.masked) {
    w.bad = take(b * p.Hk * nkt * sizeof(uint4));
    w.copy = take(b * p.Sk * p.Hk * kHeadDim * 2);
  }
  if (L.splits > 1) {
    const size_t rows = b * p.Hq * p.Sq * static_cast<size_t>(L.splits);
    w.part_o = take(rows * kHeadDim * sizeof(float));
    w.part_lse = take(rows * sizeof(float));
  }
  w.total = off;
  return w;
}

template <bool kCap, bool kBias, bool kFine>
vsa_status launch(const Args& a, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mvc,
                  cudaStream_t stream) {
  const auto kernel = masked_fwd_kernel<kCap, kBias, kFine>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Smem));
  if (e != cudaSuccess) return cuda_fail("vsa_masked_attn_fwd: shared memory", e);
  kernel<<<a.n_blocks * a.units * a.p.B * a.splits, kThreads, sizeof(Smem), stream>>>(a, mk, mv, mvc);
  e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK : cuda_fail("vsa_masked_attn_fwd", e);
}

}  // namespace

void plan(const Problem& p, PlanRows rows, int n_blocks, int4* range, int32_t* count, int32_t* list,
          cudaStream_t stream) {
  range_kernel<<<dim3((p.nkt + 3) / 4, p.B), 128, 0, stream>>>(p.doc_k, p.doc_k_sb, p.Sk, p.nkt, range);
  plan_kernel<<<dim3(n_blocks, p.B), 256, 0, stream>>>(p, range, rows, n_blocks, count, list);
}

void plan_keys(const Problem& p, const int4* range, int4* range_q, int32_t* count, int32_t* list, cudaStream_t stream) {
  const int nqt = tiles(p.Sq);
  range_kernel<<<dim3((nqt + 3) / 4, p.B), 128, 0, stream>>>(p.doc_q, p.doc_q_sb, p.Sq, nqt, range_q);
  plan_keys_kernel<<<dim3(p.nkt, p.B), 256, 0, stream>>>(p, range, range_q, nqt, count, list);
}

}  // namespace masked
}  // namespace vsa

using namespace vsa;
using namespace vsa::masked;

extern "C" {

vsa_status vsa_masked_attn_workspace_size(const vsa_mask* mask, int32_t B, int32_t Sq, int32_t Sk, int32_t Hq,
                                          int32_t Hk, size_t* bytes) {
  if (!bytes) return VSA_ERR_INVALID_ARG;
  Problem p;
  vsa_mask m = mask ? *mask : vsa_mask{};
  const int32_t documents = m.documents;
  if (documents != 0 && documents != 1) return VSA_ERR_INVALID_ARG;
  m.documents = 0;                                        // the tensors are not at hand yet
  const vsa_status st = check(mask ? &m : nullptr, nullptr, B, Sq, Sk, Hq, Hk, &p);
  if (st != VSA_OK) return st;
  p.documents = documents;
  p.masked |= documents;
  *bytes = workspace_of(p, layout_of(p)).total;
  return VSA_OK;
}

vsa_status vsa_masked_attn_fwd(const vsa_mask* mask, const vsa_mask_terms* terms, int32_t B, int32_t Sq, int32_t Sk,
                               const vsa_view* q, const vsa_view* k, const vsa_view* v, const vsa_view* out,
                               float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!q || !k || !v || !out) return VSA_ERR_INVALID_ARG;
  Args a{};
  vsa_status st = check(mask, terms, B, Sq, Sk, q->heads, k->heads, &a.p);
  if (st == VSA_OK) st = check_tensor(q, B, Sq, q->heads, false);
  if (st == VSA_OK) st = check_tensor(k, B, Sk, k->heads, false);
  if (st == VSA_OK) st = check_tensor(v, B, Sk, k->heads, false);
  if (st == VSA_OK) st = check_tensor(out, B, Sq, q->heads, true);
  if (st != VSA_OK) return st;
  if (reinterpret_cast<uintptr_t>(lse) % 4) return VSA_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256) return VSA_ERR_INVALID_ARG;
  const masked::Layout L = layout_of(a.p);
  const Workspace w = workspace_of(a.p, L);
  if (workspace_bytes < w.total) return VSA_ERR_WORKSPACE_TOO_SMALL;
  char* ws = static_cast<char*>(workspace);
  cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(int), stream);   // this call's status word
  if (e != cudaSuccess) return cuda_fail("vsa_masked_attn_fwd: cudaMemsetAsync", e);
  if (B == 0 || Sq == 0) return VSA_OK;
  if (!lse) return VSA_ERR_INVALID_ARG;
  a.out = static_cast<uint16_t*>(out->data);
  a.so = view_strides(out, B, Sq);
  a.lse = lse;
  const int row_blocks = static_cast<int>((static_cast<int64_t>(B) * q->heads * Sq + 7) / 8);
  if (Sk == 0) {
    empty_kernel<<<row_blocks, 256, 0, stream>>>(a);
    e = cudaGetLastError();
    return e == cudaSuccess ? VSA_OK : cuda_fail("vsa_masked_attn_fwd", e);
  }
  CUtensorMap mk, mv, mvc;
  st = make_map(&mk, k, B, Sk);
  if (st == VSA_OK) st = make_map(&mv, v, B, Sk);
  if (st != VSA_OK) return st;
  mvc = mv;
  a.q = static_cast<const uint16_t*>(q->data);
  a.sq = view_strides(q, B, Sq);
  const Strides sk = view_strides(k, B, Sk), sv = view_strides(v, B, Sk);
  a.k_h = sk.h != 0;
  a.k_b = sk.b != 0;
  a.v_h = sv.h != 0;
  a.v_b = sv.b != 0;
  a.packed = L.packed;
  a.units = L.units;
  a.rows = L.rows;
  a.n_blocks = L.n_blocks;
  a.one_tile = L.one_tile;
  a.splits = L.splits;
  a.err = reinterpret_cast<int*>(ws);
  if (L.splits > 1) {
    a.part_o = reinterpret_cast<float*>(ws + w.part_o);
    a.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  }
  if (a.p.documents) {
    int4* range = reinterpret_cast<int4*>(ws + w.range);
    a.count = reinterpret_cast<int32_t*>(ws + w.count);
    a.list = reinterpret_cast<int32_t*>(ws + w.list);
    plan(a.p, L.packed ? kPlanAll : L.one_tile ? kPlanSingle : kPlanPairs, L.n_blocks, range,
         reinterpret_cast<int32_t*>(ws + w.count), reinterpret_cast<int32_t*>(ws + w.list), stream);
  }
  if (a.p.masked) {
    a.clean_v = Clean{reinterpret_cast<uint4*>(ws + w.bad), reinterpret_cast<uint16_t*>(ws + w.copy)};
    st = make_map(&mvc, a.clean_v.copy, B, Sk, k->heads);
    if (st != VSA_OK) return st;
    scan_kernel<<<dim3(k->heads * a.p.nkt, B), kTileThreads, 0, stream>>>(static_cast<const uint16_t*>(v->data), sv, Sk,
                                                                          k->heads, a.p.nkt, a.clean_v);
  }
  e = cudaGetLastError();                                 // nothing reads marks or lists that nobody wrote
  if (e != cudaSuccess) return cuda_fail("vsa_masked_attn_fwd: lists and scan", e);
  const bool cap = a.p.cap > 0.0f, bias = a.p.slopes != nullptr;
  const auto run = [&](auto fine) {
    constexpr bool kFine = decltype(fine)::value;
    return cap ? (bias ? launch<true, true, kFine>(a, mk, mv, mvc, stream) : launch<true, false, kFine>(a, mk, mv, mvc, stream))
               : (bias ? launch<false, true, kFine>(a, mk, mv, mvc, stream) : launch<false, false, kFine>(a, mk, mv, mvc, stream));
  };
  st = L.rows <= kRows ? run(std::true_type{}) : run(std::false_type{});
  if (st != VSA_OK) return st;
  if (L.splits > 1) join_kernel<<<row_blocks, 256, 0, stream>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK : cuda_fail("vsa_masked_attn_fwd", e);
}

vsa_status vsa_masked_attn_status(const void* workspace, cudaStream_t stream) {
  if (!workspace) return VSA_ERR_INVALID_ARG;
  int32_t status = 0;
  cudaError_t e = cudaMemcpyAsync(&status, workspace, sizeof(status), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return cuda_fail("vsa_masked_attn_status", e);
  return static_cast<vsa_status>(status);
}

}  // extern "C"

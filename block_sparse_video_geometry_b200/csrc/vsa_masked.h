// Shared parts of the dense masked attention's forward and backward pass: the
// workspace's plan of visible tiles, the copies of rows with infinities or NaN,
// tensor maps and launch helpers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "vsa_internal.h"

namespace vsa {
namespace masked {

constexpr int kRows = 128;                  // rows of a query or key tile
constexpr size_t kHeader = 256;             // status word
constexpr uint32_t kTileBytes = 32768;      // 128 rows x 128 bf16: [d half][row][128 B], swizzled
constexpr uint64_t kTimeoutNs = 4000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int kMaxPositions = 1 << 24;      // 32-bit floats hold every distance

// A call's shape and mask as the kernels read them.
struct Problem {
  int32_t B, Hq, Hk, group;                 // group = Hq / Hk
  int32_t Sq, Sk, off;                      // off = Sk - Sq: key position of query 0
  int32_t nkt;                              // key tiles
  int32_t causal, documents;
  int32_t masked;                           // some pair may be invisible (rows may need clean copies)
  const int32_t *doc_q, *doc_k;
  int64_t doc_q_sb, doc_k_sb;
  const int32_t* prefix;
  const float* slopes;
  float scale, cap;

  // Last key position that query i sees by order.
  __device__ __forceinline__ int limit(int b, int i) const {
    if (!causal) return Sk - 1;
    const int p = prefix ? max(prefix[b], 0) : 0;          // any 32-bit value
    return min(max(i + off, p - 1), Sk - 1);
  }
};

// Rows of a tensor that hold an infinity or NaN, per 128-row tile, and copies of
// those tiles with such rows zeroed: a product over a tile multiplies masked
// entries by 0, which must not meet one.
struct Clean {
  uint4* bad;                               // [B][heads][tiles] bit r: row r of the tile is bad; null: not scanned
  uint16_t* copy;                           // [B][S][heads][128]; only tiles with a bad row are written
};

inline int tiles(int n) { return (n + kRows - 1) / kRows; }

#ifdef __CUDACC__
constexpr int kTileThreads = 256;           // threads that hold a tile: 8 pieces of 16 bytes each
constexpr int kPieces = 8;

// Piece i of thread t is row (256 i + t) / 16, channels 8 ((256 i + t) % 16) ..+7; rows past n: zero.
__device__ __forceinline__ void load_pieces(uint4 (&w)[kPieces], const uint16_t* base, int64_t row_stride, int n) {
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int e = i * kTileThreads + threadIdx.x, r = e >> 4;
    w[i] = make_uint4(0, 0, 0, 0);
    if (r < n) w[i] = *reinterpret_cast<const uint4*>(base + r * row_stride + (e & 15) * 8);
  }
}

// Marks the rows of the block's tile that hold an infinity or NaN (bad[4], cleared).
__device__ __forceinline__ void find_bad(const uint4 (&w)[kPieces], uint32_t* bad) {
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int r = (i * kTileThreads + threadIdx.x) >> 4;
    bool any = false;
    for (uint32_t v : {w[i].x, w[i].y, w[i].z, w[i].w})
      any |= (v & 0x7F80u) == 0x7F80u || (v & 0x7F800000u) == 0x7F800000u;
    if (any) atomicOr(&bad[r >> 5], 1u << (r & 31));
  }
}

// Behind a barrier: the tile's marks, and its copy without such rows if there are any.
__device__ __forceinline__ void write_clean(const Clean& c, uint4 (&w)[kPieces], const uint32_t* bad, int b, int h,
                                            int heads, int tile, int n_tiles, int S) {
  const uint4 m = make_uint4(bad[0], bad[1], bad[2], bad[3]);
  if (threadIdx.x == 0) c.bad[(static_cast<size_t>(b) * heads + h) * n_tiles + tile] = m;
  if (!(m.x | m.y | m.z | m.w)) return;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int e = i * kTileThreads + threadIdx.x, r = e >> 4;
    if (tile * kRows + r >= S) continue;
    if ((bad[r >> 5] >> (r & 31)) & 1u) w[i] = make_uint4(0, 0, 0, 0);
    const size_t row = (static_cast<size_t>(b) * S + tile * kRows + r) * heads + h;
    *reinterpret_cast<uint4*>(c.copy + row * kHeadDim + (e & 15) * 8) = w[i];
  }
}
#endif

// cuTensorMapEncodeTiled over a view: boxes of 64 channels x 128 rows of one
// head and batch entry, 128-byte swizzled, rows past S read as zero.
vsa_status make_map(CUtensorMap* map, const vsa_view* v, int32_t B, int32_t S);
vsa_status make_map(CUtensorMap* map, const uint16_t* copy, int32_t B, int32_t S, int32_t heads);

// Validation shared by both passes; fills `p`.
vsa_status check(const vsa_mask* mask, const vsa_mask_terms* t, int32_t B, int32_t Sq, int32_t Sk, int32_t Hq,
                 int32_t Hk, Problem* p);
vsa_status check_tensor(const vsa_view* v, int32_t B, int32_t S, int32_t heads, bool output);

// Records of a list of visible tiles: the tile, whether it holds one document only,
// and whether documents hide part of it from query tile 0 or 1 of the block.
constexpr int kOneDoc = 1 << 28, kPartial0 = 1 << 29, kPartial1 = 1 << 30, kTileMask = kOneDoc - 1;

// Visible key tiles of query blocks (documents only). `range`: [B][nkt] scratch;
// count [B][n_blocks], list [B][n_blocks][nkt] out.
enum PlanRows { kPlanPairs, kPlanAll, kPlanSingle };   // two tiles a block, all queries in one block, one tile a block
void plan(const Problem& p, PlanRows rows, int n_blocks, int4* range, int32_t* count, int32_t* list,
          cudaStream_t stream);
// Visible query tiles of key tiles: range_q [B][nqt] scratch, `range` filled by
// plan(); count [B][nkt], list [B][nkt][nqt] out.
void plan_keys(const Problem& p, const int4* range, int4* range_q, int32_t* count, int32_t* list, cudaStream_t stream);

}  // namespace masked
}  // namespace vsa

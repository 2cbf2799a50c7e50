// Rotary positions with three axes (time, height, width) for q and k, and the
// gradient (the rotation by the negative angle).
//
// Mathematics: y_a = x_a cos - x_b sin, y_b = x_a sin + x_b cos for the pairs
// (a, b) of each axis' channel block, angle = pos * scale * theta^(-2i/dim). A
// 32-bit angle of a far position is off by pos * 2^-24 radians (0.06 at 10^6),
// so the host gives each pair's rate in turns per position in 64 bits and the
// kernel keeps only the fraction of a turn: t = pos * rate, t - round(t), whose
// sine and cosine are 32-bit functions of a value in [-1/2, 1/2].
//
// Bound: HBM (one read and one write of q and k; 12 bytes of position a token).
// One block takes a few tokens: its threads compute the tokens' 64 sines and
// cosines once into shared memory, shared by all heads of q and k, then stream
// the heads' rows in chunks of 8 channels, two chunks in flight per thread. Measured:
// 133,696 tokens x 48 heads, bf16 538 us (93% of the copy rate).
// A chunk holds whole pairs when pairs are adjacent; with halves the partner
// channels sit in other chunks of the row at offsets that need not be multiples
// of 8 (a width block of 42 channels), so the 16 lanes of a row exchange them
// through shared memory; where every axis' dim is a multiple of 8, a lane takes four
// pairs with both their channels instead, in two accesses of four (133,696 tokens x 48
// heads, bf16: 762 us exchanging, 547 us so; fp32 to bf16, 17,408 x 32 heads: 96 and 80).

#include <cmath>

#include "vec.cuh"
#include "vsa_internal.h"

namespace vsa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kPairs = kHeadDim / 2;
constexpr int kChunk = 8;                        // channels per thread and step
constexpr int kLanes = kHeadDim / kChunk;        // lanes per row
constexpr int kRopeUnroll = 2;                   // rows in flight per thread
constexpr int kRopeTokens = 16;                  // most tokens per block
constexpr int kRopeMaxHeads = 4096;              // of q and of k: row numbers of a block times heads fit 32 bits

struct RopeTable {
  double rate[kPairs];         // turns per position
  int32_t rotated;             // channels before the pass-through ones
  uint8_t axis[kPairs];
  uint8_t a[kPairs], b[kPairs];   // the pair's channels: y_a = x_a cos - x_b sin, y_b = x_b cos + x_a sin
  // channel -> its partner's place in a shared-memory row (bits 0-7), kPass where it is not rotated
  uint32_t channel[kHeadDim];
};
constexpr uint32_t kPass = 1u << 16;

struct RopeArgs {
  const void* in[2];
  void* out[2];
  Strides si[2], so[2];
  int heads_q, heads;          // heads of q, and of q and k together
  uint64_t per_head;           // ceil(2^32 / heads): rows of a block / heads by one multiplication
  int64_t n_tokens, S;
  const int32_t* pos;
  int64_t pos_sb;
  float sign;                  // +1 forward, -1 backward
};

// Shared memory holds a row of 128 channels as [i][lane] for channel 8 lane + i,
// padded so that neither the writes nor the partner's reads of a warp's two rows
// meet in a bank (in channel order they met eight at a time: 195 us for the fp32
// gradient of 17,408 x 32 heads).
constexpr int kRowPitch = kLanes + 1, kRowWords = 144;
__host__ __device__ __forceinline__ int row_word(int channel) { return channel % kChunk * kRowPitch + channel / kChunk; }

enum RopeForm { kAdjacent, kExchange, kQuads };

template <class I, class O, RopeForm kForm>
__global__ void __launch_bounds__(kRopeThreads, kForm == kExchange ? 4 : 6)
rope_kernel(const __grid_constant__ RopeTable tab, const __grid_constant__ RopeArgs a, int tokens_per_block) {
  constexpr bool kHalves = kForm == kExchange;
  extern __shared__ float2 turn[];               // [token][row_word(channel)] or [token][pair]: cos, signed sin
  __shared__ int64_t base[kRopeTokens][4];       // element offset of each token in q, k and their outputs
  __shared__ float rows[kHalves ? kRopeThreads / kLanes * kRowWords : 1];
  constexpr int kTurns = kHalves ? kRowWords : kPairs;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tokens_per_block;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens_per_block), a.n_tokens - t0));
  if (threadIdx.x < 4 * nt) {
    const int p = threadIdx.x & 3;
    const uint32_t tok = static_cast<uint32_t>(t0) + threadIdx.x / 4, S = static_cast<uint32_t>(a.S);   // < 2^31
    const int64_t b = tok / S, s = tok - static_cast<uint32_t>(b) * S;
    const Strides st = p == 0 ? a.si[0] : p == 1 ? a.si[1] : p == 2 ? a.so[0] : a.so[1];
    base[threadIdx.x / 4][p] = b * st.b + s * st.s;
  }
  const int lane = threadIdx.x % kLanes, c0 = lane * kChunk;
  // Values of the parameter block at an index that differs between lanes are read
  // one lane after the other: each thread reads its own once per block.
  uint32_t ch[kHalves ? kChunk : 1];
  if constexpr (kHalves) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      ch[i] = tab.channel[c0 + i];
      asm volatile("" : "+r"(ch[i]));            // held: not to be read again from the parameters
    }
  }
  uint32_t qa = 0, qb = 0;                       // kQuads: the first channels of the lane's pairs
  if constexpr (kForm == kQuads) {
    qa = tab.a[4 * lane];
    qb = tab.b[4 * lane];
    asm volatile("" : "+r"(qa), "+r"(qb));
  }
  const int pr = threadIdx.x % kPairs;
  const double rate = tab.rate[pr];
  const int axis = tab.axis[pr];
  const int ca = kHalves ? row_word(tab.a[pr]) : 0, cb = kHalves ? row_word(tab.b[pr]) : 0;
  __syncthreads();

  const int group = threadIdx.x / kLanes;
  constexpr int kGroups = kRopeThreads / kLanes;
  const int n_rows = nt * a.heads;
  constexpr int kPiece = kForm == kQuads ? 4 : kChunk;
  Pack<I, kPiece> x[kRopeUnroll], xb[kForm == kQuads ? kRopeUnroll : 1];
  O* dst[kRopeUnroll];
  int tk[kRopeUnroll];
  // Every lane runs every step (the exchange synchronises warps); rows past the
  // end are neither read nor written.
  auto fetch = [&](int row0) {
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const int r = row0 + u * kGroups + group;
      dst[u] = nullptr;
      tk[u] = 0;
      if (r >= n_rows) continue;
      tk[u] = static_cast<int>(static_cast<uint32_t>(r) * a.per_head >> 32);
      const int hh = r - tk[u] * a.heads;
      const bool w = hh >= a.heads_q;
      const int64_t h = w ? hh - a.heads_q : hh;
      const int64_t* at = base[tk[u]] + w;
      const I* src = static_cast<const I*>(w ? a.in[1] : a.in[0]) + at[0] + h * (w ? a.si[1].h : a.si[0].h);
      dst[u] = static_cast<O*>(w ? a.out[1] : a.out[0]) + at[2] + h * (w ? a.so[1].h : a.so[0].h);
      if constexpr (kForm == kQuads) {
        x[u].load(src + qa);
        xb[u].load(src + qb);
      } else {
        x[u].load(src + c0);
        dst[u] += c0;
      }
    }
  };
  for (int i = threadIdx.x / kPairs; i < nt; i += kRopeThreads / kPairs) {
    const uint32_t tok = static_cast<uint32_t>(t0) + i, S = static_cast<uint32_t>(a.S);
    const int64_t b = tok / S, s = tok - static_cast<uint32_t>(b) * S;
    const double t = static_cast<double>(a.pos[b * a.pos_sb + 3 * s + axis]) * rate;
    float sn, cs;
    sincospif(2.0f * static_cast<float>(t - rint(t)), &sn, &cs);
    sn *= a.sign;
    float2* tt = turn + i * kTurns;
    if constexpr (kHalves) {
      tt[ca] = make_float2(cs, -sn);
      tt[cb] = make_float2(cs, sn);
    } else {
      tt[pr] = make_float2(cs, sn);
    }
  }
  __syncthreads();

  for (int row0 = 0; row0 < n_rows; row0 += kGroups * kRopeUnroll) {
    fetch(row0);
#pragma unroll
    for (int u = 0; u < kRopeUnroll; ++u) {
      const float2* tt = turn + tk[u] * kTurns;
      if constexpr (kForm == kQuads) {
        if (!dst[u]) continue;
        float p[4], q[4], ya[4], yb[4];
        x[u].get(p);
        xb[u].get(q);
        const bool pass = 8 * lane >= tab.rotated;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 cs = tt[4 * lane + i];
          ya[i] = pass ? p[i] : fmaf(p[i], cs.x, -q[i] * cs.y);
          yb[i] = pass ? q[i] : fmaf(q[i], cs.x, p[i] * cs.y);
        }
        Pack<O, 4> o;
        o.set(ya);
        o.store(dst[u] + qa);
        o.set(yb);
        o.store(dst[u] + qb);
        continue;
      }
      float v[kChunk], y[kChunk];
      if constexpr (kHalves) {
        float* row = rows + group * kRowWords;
        if (dst[u]) {
          x[u].get(v);
#pragma unroll
          for (int i = 0; i < kChunk; ++i) row[i * kRowPitch + lane] = v[i];
        }
        __syncwarp();
        if (dst[u]) {
#pragma unroll
          for (int i = 0; i < kChunk; ++i) {
            const float2 cs = tt[i * kRowPitch + lane];
            const float z = fmaf(v[i], cs.x, row[ch[i] & 0xFFu] * cs.y);
            y[i] = ch[i] & kPass ? v[i] : z;
          }
        }
        __syncwarp();
      } else if constexpr (kForm == kAdjacent) {
        if (!dst[u]) continue;
        x[u].get(v);
#pragma unroll
        for (int i = 0; i < kChunk; i += 2) {
          const float2 cs = tt[(c0 + i) / 2];
          const float za = fmaf(v[i], cs.x, -v[i + 1] * cs.y);
          const float zb = fmaf(v[i + 1], cs.x, v[i] * cs.y);
          y[i] = c0 + i >= tab.rotated ? v[i] : za;
          y[i + 1] = c0 + i >= tab.rotated ? v[i + 1] : zb;
        }
      }
      if (dst[u]) {
        Pack<O, kChunk> o;
        o.set(y);
        o.store(dst[u]);
      }
    }
  }
}

// Token positions of a layout: conditioning tokens counted along the sequence,
// video tokens by their place in the grid.
__global__ void __launch_bounds__(256)
rope_positions_kernel(int64_t seq_len, int64_t video_start, int64_t video_len, int grid_h, int grid_w, int t0, int h0,
                      int w0, int32_t* __restrict__ pos) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= seq_len) return;
  const int64_t n = i - video_start;
  uint32_t p[3];
  if (n >= 0 && n < video_len) {
    const int64_t hw = static_cast<int64_t>(grid_h) * grid_w;
    p[0] = static_cast<uint32_t>(t0) + static_cast<uint32_t>(n / hw);
    p[1] = static_cast<uint32_t>(h0) + static_cast<uint32_t>(n % hw / grid_w);
    p[2] = static_cast<uint32_t>(w0) + static_cast<uint32_t>(n % grid_w);
  } else {
    p[0] = p[1] = p[2] = static_cast<uint32_t>(n < 0 ? i : i - video_len);
  }
  for (int a = 0; a < 3; ++a) pos[3 * i + a] = static_cast<int32_t>(p[a]);
}

// Turn rates and channel pairing of a vsa_rope; false when it is malformed.
bool rope_table(const vsa_rope* r, RopeTable* t) {
  if (!r || (r->pairing != VSA_ROPE_ADJACENT && r->pairing != VSA_ROPE_HALVES)) return false;
  if (!(r->theta > 0.0) || !std::isfinite(r->theta)) return false;
  const int64_t dim[3] = {r->dim_t, r->dim_h, r->dim_w};
  const double scale[3] = {r->scale_t, r->scale_h, r->scale_w};
  int64_t sum = 0;
  for (int ax = 0; ax < 3; ++ax) {
    if (dim[ax] < 0 || dim[ax] % 2 || !std::isfinite(scale[ax])) return false;
    sum += dim[ax];
  }
  if (sum > kHeadDim) return false;
  t->rotated = static_cast<int32_t>(sum);
  constexpr double kTwoPi = 6.283185307179586476925;
  for (int p = 0; p < kPairs; ++p) {             // pass through unless set below
    t->rate[p] = 0.0;
    t->axis[p] = 0;
  }
  int at = 0;
  const bool halves = r->pairing == VSA_ROPE_HALVES;
  const int dims4[4] = {r->dim_t, r->dim_h, r->dim_w, static_cast<int>(kHeadDim - sum)};
  for (int ax = 0; ax < 4; ++ax) {
    const int d = dims4[ax];
    for (int i = 0; i < d / 2; ++i) {
      const int p = at / 2 + i;
      if (ax < 3) {
        t->rate[p] = std::pow(r->theta, -2.0 * i / d) * scale[ax] / kTwoPi;
        if (!std::isfinite(t->rate[p])) return false;
        t->axis[p] = static_cast<uint8_t>(ax);
      }
      const int ca = at + (halves ? i : 2 * i), cb = halves ? ca + d / 2 : ca + 1;
      const uint32_t pass = ax == 3 ? kPass : 0u;
      t->a[p] = static_cast<uint8_t>(ca);
      t->b[p] = static_cast<uint8_t>(cb);
      t->channel[ca] = pass | static_cast<uint32_t>(row_word(cb));
      t->channel[cb] = pass | static_cast<uint32_t>(row_word(ca));
    }
    at += d;
  }
  return true;
}

template <class I, class O>
void rope_launch(const RopeTable& tab, const RopeArgs& a, RopeForm form, int tpb, int blocks, cudaStream_t stream) {
  const size_t smem = sizeof(float2) * (form == kExchange ? kRowWords : kPairs) * tpb;
  if (form == kExchange)
    rope_kernel<I, O, kExchange><<<blocks, kRopeThreads, smem, stream>>>(tab, a, tpb);
  else if (form == kQuads)
    rope_kernel<I, O, kQuads><<<blocks, kRopeThreads, smem, stream>>>(tab, a, tpb);
  else
    rope_kernel<I, O, kAdjacent><<<blocks, kRopeThreads, smem, stream>>>(tab, a, tpb);
}

template <class I>
void rope_launch_in(int out, const RopeTable& tab, const RopeArgs& a, RopeForm form, int tpb, int blocks,
                    cudaStream_t stream) {
  if (out == VSA_F32) rope_launch<I, float>(tab, a, form, tpb, blocks, stream);
  else if (out == VSA_BF16) rope_launch<I, bf16>(tab, a, form, tpb, blocks, stream);
  else rope_launch<I, f16>(tab, a, form, tpb, blocks, stream);
}

vsa_status rope_call(const char* where, const vsa_rope* rope, int32_t B, int64_t S, const int32_t* pos, int64_t pos_sb,
                     const vsa_view* q, const vsa_view* k, const vsa_view* q_out, const vsa_view* k_out, float sign,
                     cudaStream_t stream) {
  RopeTable tab;
  if (!rope_table(rope, &tab) || B < 0 || S < 0) return VSA_ERR_INVALID_ARG;
  if (!q || !q_out || (k == nullptr) != (k_out == nullptr)) return VSA_ERR_INVALID_ARG;
  const vsa_view* in[2] = {q, k};
  const vsa_view* out[2] = {q_out, k_out};
  for (int w = 0; w < (k ? 2 : 1); ++w) {
    vsa_status st = check_view(in[w], B, S, kHeadDim, 16, false);
    if (st == VSA_OK) st = check_view(out[w], B, S, kHeadDim, 16, true);
    if (st != VSA_OK) return st;
    if (in[w]->heads != out[w]->heads) return VSA_ERR_INVALID_ARG;
    if (in[w]->heads > kRopeMaxHeads) return VSA_ERR_UNSUPPORTED;
  }
  if (B == 0 || S == 0) return VSA_OK;
  if (!pos || reinterpret_cast<uintptr_t>(pos) % 4) return VSA_ERR_INVALID_ARG;
  if (B > 1 && pos_sb != 0 && (pos_sb < 0 || pos_sb / 3 < S || pos_sb > INT64_MAX / 16 / B)) return VSA_ERR_INVALID_ARG;
  if (S > INT32_MAX / B) return VSA_ERR_UNSUPPORTED;

  // q and k in one launch where they have the same types, else one launch each.
  const bool together = k && q->dtype == k->dtype && q_out->dtype == k_out->dtype;
  for (int w = 0; w < (k && !together ? 2 : 1); ++w) {
    RopeArgs a{};
    for (int i = 0; i < 2; ++i) {
      const int src = together ? i : w;
      a.in[i] = in[src]->data;
      a.out[i] = out[src]->data;
      a.si[i] = view_strides(in[src], B, S);
      a.so[i] = view_strides(out[src], B, S);
    }
    a.heads_q = in[w]->heads;
    a.heads = together ? q->heads + k->heads : in[w]->heads;
    a.per_head = ((uint64_t{1} << 32) + a.heads - 1) / a.heads;
    a.S = S;
    a.n_tokens = S * B;
    a.pos = pos;
    a.pos_sb = B > 1 ? pos_sb : 0;
    a.sign = sign;
    const int tpb = a.n_tokens >= 8192 ? kRopeTokens : a.n_tokens >= 2048 ? 4 : 1;
    const int blocks = static_cast<int>((a.n_tokens + tpb - 1) / tpb);
    // dims of multiples of 8: the halves of every axis start at multiples of 4 channels
    const RopeForm form = rope->pairing != VSA_ROPE_HALVES                                  ? kAdjacent
                          : rope->dim_t % 8 == 0 && rope->dim_h % 8 == 0 && rope->dim_w % 8 == 0 ? kQuads
                                                                                            : kExchange;
    if (in[w]->dtype == VSA_F32) rope_launch_in<float>(out[w]->dtype, tab, a, form, tpb, blocks, stream);
    else if (in[w]->dtype == VSA_BF16) rope_launch_in<bf16>(out[w]->dtype, tab, a, form, tpb, blocks, stream);
    else rope_launch_in<f16>(out[w]->dtype, tab, a, form, tpb, blocks, stream);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(where, e);
  }
  return VSA_OK;
}

}  // namespace
}  // namespace vsa

using namespace vsa;

extern "C" {

vsa_status vsa_rope_positions(const vsa_layout* L, int32_t t0, int32_t h0, int32_t w0, int32_t* pos,
                              cudaStream_t stream) {
  if (!L || !pos || reinterpret_cast<uintptr_t>(pos) % 4) return VSA_ERR_INVALID_ARG;
  const int64_t n_video = static_cast<int64_t>(L->grid_t) * L->grid_h * L->grid_w;
  const int blocks = static_cast<int>((L->seq_len + 255) / 256);
  rope_positions_kernel<<<blocks, 256, 0, stream>>>(L->seq_len, L->video_start, n_video, L->grid_h, L->grid_w, t0, h0,
                                                    w0, pos);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VSA_OK : cuda_fail("vsa_rope_positions", e);
}

vsa_status vsa_rope_fwd(const vsa_rope* rope, int32_t B, int64_t S, const int32_t* pos, int64_t pos_stride_b,
                        const vsa_view* q, const vsa_view* k, const vsa_view* q_out, const vsa_view* k_out,
                        cudaStream_t stream) {
  return rope_call("vsa_rope_fwd", rope, B, S, pos, pos_stride_b, q, k, q_out, k_out, 1.0f, stream);
}

vsa_status vsa_rope_bwd(const vsa_rope* rope, int32_t B, int64_t S, const int32_t* pos, int64_t pos_stride_b,
                        const vsa_view* dq_out, const vsa_view* dk_out, const vsa_view* dq, const vsa_view* dk,
                        cudaStream_t stream) {
  return rope_call("vsa_rope_bwd", rope, B, S, pos, pos_stride_b, dq_out, dk_out, dq, dk, -1.0f, stream);
}

}  // extern "C"

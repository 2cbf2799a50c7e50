// Loads and stores of a few consecutive elements of a storage type (float,
// bf16, fp16) as 32-bit floats.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace vsa {

using bf16 = __nv_bfloat16;
using f16 = __half;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(f16 x) { return __half2float(x); }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ f16 from_f32<f16>(float x) { return __float2half_rn(x); }

// N consecutive elements in as few words as they fill (N * sizeof(T) is a
// multiple of the word: 16, 8 or 4 bytes, or one element).
template <class T, int N>
struct Pack {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T));
  static constexpr int kWord = kBytes % 16 == 0 ? 16 : kBytes % 8 == 0 ? 8 : kBytes % 4 == 0 ? 4 : 2;
  union {
    T t[N];
    uint4 u4[kBytes >= 16 ? kBytes / 16 : 1];
    uint2 u2;
    uint32_t u1;
    uint16_t h;
  };
  __device__ __forceinline__ Pack() {}
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWord == 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) u4[i] = reinterpret_cast<const uint4*>(p)[i];
    } else if constexpr (kWord == 8) {
      u2 = *reinterpret_cast<const uint2*>(p);
    } else if constexpr (kWord == 4) {
      u1 = *reinterpret_cast<const uint32_t*>(p);
    } else {
      h = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWord == 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(p)[i] = u4[i];
    } else if constexpr (kWord == 8) {
      *reinterpret_cast<uint2*>(p) = u2;
    } else if constexpr (kWord == 4) {
      *reinterpret_cast<uint32_t*>(p) = u1;
    } else {
      *reinterpret_cast<uint16_t*>(p) = h;
    }
  }
  __device__ __forceinline__ void get(float (&x)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(t[i]);
  }
  __device__ __forceinline__ void set(const float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) t[i] = from_f32<T>(x[i]);
  }
};

}  // namespace vsa

// Loads and stores of a few consecutive elements of a storage type (float,
// bf16, fp16) as 32-bit floats.
#pragma once

#include <cstdint>
#include <type_traits>
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

// N consecutive elements in words of the widest access that fills them (16, 8, 4
// or 2 bytes); as large as the elements.
template <class T, int N>
struct Pack {
  static constexpr int kBytes = N * static_cast<int>(sizeof(T));
  using Word = std::conditional_t<
      kBytes % 16 == 0, uint4,
      std::conditional_t<kBytes % 8 == 0, uint2, std::conditional_t<kBytes % 4 == 0, uint32_t, uint16_t>>>;
  static constexpr int kWords = kBytes / static_cast<int>(sizeof(Word));
  union {
    T t[N];
    Word w[kWords];
  };
  __device__ __forceinline__ Pack() {}
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const Word*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<Word*>(p)[i] = w[i];
  }
  __device__ __forceinline__ void get(float (&x)[N]) const {
    if constexpr (sizeof(T) == 2 && sizeof(Word) > 2 && std::is_same_v<T, bf16>) {
      // bf16 is the upper half of a float
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const uint32_t p = reinterpret_cast<const uint32_t*>(w)[i / 2];
        x[i] = __uint_as_float(p << 16);
        x[i + 1] = __uint_as_float(p & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = to_f32(t[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[N]) {
    if constexpr (sizeof(T) == 2 && sizeof(Word) > 2) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        if constexpr (std::is_same_v<T, bf16>)
          reinterpret_cast<__nv_bfloat162*>(w)[i / 2] = __floats2bfloat162_rn(x[i], x[i + 1]);
        else
          reinterpret_cast<__half2*>(w)[i / 2] = __floats2half2_rn(x[i], x[i + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = from_f32<T>(x[i]);
    }
  }
};

// Element-wise arithmetic on N floats, two per instruction where N is even.
template <int N, class F2, class F1>
__device__ __forceinline__ void each(F2 two, F1 one) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) two(i);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) one(i);
  }
}

static_assert(sizeof(Pack<float, 1>) == 4 && sizeof(Pack<bf16, 1>) == 2 && sizeof(Pack<bf16, 8>) == 16);

}  // namespace vsa

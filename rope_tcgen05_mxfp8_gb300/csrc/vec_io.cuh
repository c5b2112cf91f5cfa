// Element types of the block operators (bf16, fp16, fp32) as vectors: loads and stores of
// N consecutive elements as one access, conversions to and from fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace qkvcte {

// N elements of T moved as one access (16 bytes at most): the address must be a multiple
// of N * sizeof(T).
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  static_assert(sizeof(T) * N <= 16, "one access");
  T v[N];
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// Round to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
  return __float2half_rn(x);
}

// Data read once: past L1, whose lines stay with what is read again (parameters). Not the
// read-only path: the caller may write the same elements in place afterwards.
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> ld_once(const T* p) {
  Vec<T, N> r;
  if constexpr (sizeof(r) == 16) {
    uint32_t w[4];
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p)
                 : "memory");
    r = *reinterpret_cast<Vec<T, N>*>(w);
  } else {
    r = *reinterpret_cast<const Vec<T, N>*>(p);
  }
  return r;
}

template <typename T, int N>
__device__ __forceinline__ void st_vec(T* p, const Vec<T, N>& r) {
  *reinterpret_cast<Vec<T, N>*>(p) = r;
}

// N parameters starting at p (16-byte aligned when N > 1), as fp32.
template <typename P, int N>
__device__ __forceinline__ void ld_params(const P* p, float* out) {
  constexpr int PN = 16 / sizeof(P) < N ? 16 / sizeof(P) : N;
#pragma unroll
  for (int i = 0; i < N; i += PN) {
    const Vec<P, PN> r = *reinterpret_cast<const Vec<P, PN>*>(p + i);
#pragma unroll
    for (int j = 0; j < PN; ++j) out[i + j] = to_f32(r.v[j]);
  }
}

}  // namespace qkvcte

// Element types of the block operators (bf16, fp16, fp32) as vectors: loads and stores of
// N consecutive elements as one access, conversions to and from fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace qkvcte {

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

// Two packed 2-byte elements (the first in the low half) and fp32 pairs.
template <typename T>
__device__ __forceinline__ float2 unpack_pair(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack_pair<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 unpack_pair<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float2 v);
template <>
__device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float2 v) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&p);
}
template <>
__device__ __forceinline__ uint32_t pack_pair<__half>(float2 v) {
  const __half2 p = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// N elements of T moved as one access (16 bytes at most): the address must be a multiple
// of N * sizeof(T). Held as 32-bit words (as elements, the compiler takes 16-bit lanes
// apart and puts them together again around every use); read and written in pairs, or as
// the one element there is.
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
  static_assert(sizeof(T) * N >= 4 && sizeof(T) * N <= 16 && N % 2 == 0, "whole words in one access");
  uint32_t w[sizeof(T) * N / 4];

  __device__ __forceinline__ float2 pair(int j) const {
    if constexpr (sizeof(T) == 4)
      return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    else
      return unpack_pair<T>(w[j]);
  }
  __device__ __forceinline__ void set_pair(int j, float2 v) {
    if constexpr (sizeof(T) == 4) {
      w[2 * j] = __float_as_uint(v.x);
      w[2 * j + 1] = __float_as_uint(v.y);
    } else {
      w[j] = pack_pair<T>(v);
    }
  }
};

template <typename T>
struct Vec<T, 1> {
  T v;
  __device__ __forceinline__ float one() const { return to_f32(v); }
  __device__ __forceinline__ void set_one(float x) { v = from_f32<T>(x); }
};

// Data read once: past L1, whose lines stay with what is read again. Not the read-only
// path: the caller may write the same elements in place afterwards.
template <typename T, int N>
__device__ __forceinline__ Vec<T, N> ld_once(const T* p) {
  Vec<T, N> r;
  if constexpr (sizeof(r) == 16) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p)
                 : "memory");
  } else {
    r = *reinterpret_cast<const Vec<T, N>*>(p);
  }
  return r;
}

template <typename T, int N>
__device__ __forceinline__ void st_vec(T* p, const Vec<T, N>& r) {
  *reinterpret_cast<Vec<T, N>*>(p) = r;
}

// 16-byte asynchronous copy to a shared address, past L1 (the thread's own copies, by
// groups), and a 16-byte read of it.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ld_shared16(uint32_t src, uint32_t* w) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(src)
               : "memory");
}
// One element at a shared address.
template <typename T>
__device__ __forceinline__ T ld_shared_elem(uint32_t src) {
  T r;
  if constexpr (sizeof(T) == 4) {
    uint32_t w;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(src) : "memory");
    r = *reinterpret_cast<T*>(&w);
  } else {
    uint16_t w;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(src) : "memory");
    r = *reinterpret_cast<T*>(&w);
  }
  return r;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace qkvcte

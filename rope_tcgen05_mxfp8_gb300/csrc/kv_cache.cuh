// Device helpers of the 8-bit key/value cache: pages, scales and codes.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "kv_cache.h"

namespace qkvcte {

constexpr int kScaleNan = 255;  // UE8M0: a page and head that hold a value that is not finite

// The table's entry for block `blk` of sequence b, -1 behind the table. (Without a table
// b * max_blocks + blk < pages, which fits.)
__device__ __forceinline__ int cache_entry(const CachePool& p, int b, long long blk) {
  if (blk < 0 || blk >= p.max_blocks) return -1;
  return p.table != nullptr ? __ldg(p.table + b * p.table_stride + blk) : b * p.max_blocks + static_cast<int>(blk);
}

// The page of that block, or -1: also for a hole (an entry that is no page of the pool). Every
// access to the pool is by a page that was checked so.
__device__ __forceinline__ long long cache_page(const CachePool& p, int b, long long blk) {
  const int page = cache_entry(p, b, blk);
  return page >= 0 && page < p.pages ? page : -1;
}

// 2^(e - 127); NaN for 255.
__device__ __forceinline__ float scale_value(int e) {
  const uint32_t bits = e == 0 ? 0x00400000u : e >= kScaleNan ? 0x7FC00000u : static_cast<uint32_t>(e) << 23;
  return __uint_as_float(bits);
}

// Biased exponent E of the smallest power of two 2^(E - 127) that brings |x| to at most
// 448 = 1.75 * 2^8, from x's bits without the sign: 1 (the least) for zeros, 255 for
// infinities and NaN.
__device__ __forceinline__ int scale_exponent(uint32_t abs_bits) {
  if (abs_bits >= 0x7F800000u) return kScaleNan;
  const int e = static_cast<int>(abs_bits >> 23) - 8 + ((abs_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < 1 ? 1 : e;
}

// 16 codes, zeros without `live` (nothing is read then). One predicated instruction: a branch
// around each load made the next ones wait for it.
__device__ __forceinline__ uint4 ld_codes_if(const uint8_t* p, bool live) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@q ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(static_cast<int>(live)));
  return v;
}

// Two e4m3 codes (the low 16 bits) as fp16, exactly.
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(codes));
  return h;
}
// The upper two of four codes.
__device__ __forceinline__ uint32_t codes_hi_to_half2(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(codes));
  return h;
}

__device__ __forceinline__ float2 half2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// fp32 pair -> e4m3 codes (x in the low byte), to nearest even, saturating.
__device__ __forceinline__ uint32_t f32_to_codes(float x, float y) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(y), "f"(x));  // the first source is the upper byte
  return c;
}

// Tokens of sequence b that a query row may see, as the kernels walk them: positions
// [lo, hi) (empty: hi <= lo).
struct Visible {
  int length, first_pos;  // first_pos: of query 0 (may be negative)
  int count;

  __device__ __forceinline__ Visible(const CacheAttentionArgs& a, int b) {
    const long long cap = static_cast<long long>(a.pool.max_blocks) << a.pool.log_bt;
    const int n = __ldg(a.lengths + b);
    length = n < 0 ? 0 : n > cap ? static_cast<int>(cap) : n;
    const int c = a.counts != nullptr ? __ldg(a.counts + b) : a.seq;
    count = c < 0 ? 0 : c > a.seq ? a.seq : c;
    first_pos = length - count;
  }
  __device__ __forceinline__ int hi(const CacheAttentionArgs& a, int s) const {
    if (s >= count) return 0;
    const int pos = first_pos + s;
    return !a.causal ? length : pos + 1 > 0 ? pos + 1 : 0;  // pos < length
  }
  __device__ __forceinline__ int lo(const CacheAttentionArgs& a, int s) const {
    if (a.window == 0) return 0;
    const long long first = static_cast<long long>(first_pos) + s - a.window + 1;
    return first > 0 ? static_cast<int>(first) : 0;
  }
};

// A row of queries in fp16: scaled by a power of two so that its largest element lies in
// [2^14, 2^15), which loses nothing of bf16's or fp16's digits but in elements 2^-28 of the
// largest. Returns the exponent field of the factor from the bits of the largest element.
__device__ __forceinline__ int query_factor_field(uint32_t abs_bits) {
  const int f = 268 - static_cast<int>(abs_bits >> 23);
  return f > 253 ? 253 : f;
}
// What brings a row's products back and scales them; NaN for a row with an element that is not
// finite: infinite scores alone, all of one sign, would pass for a row that sees nothing.
__device__ __forceinline__ float query_coef(uint32_t abs_bits, int field, float scale_log2) {
  return scale_log2 * scale_value(abs_bits >= 0x7F800000u ? kScaleNan : 254 - field);
}

}  // namespace qkvcte

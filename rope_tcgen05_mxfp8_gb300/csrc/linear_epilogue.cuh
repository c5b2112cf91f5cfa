// The product's epilogue: O = residual + gate * act(z), z = acc * scale + bias, on 16
// columns of one row at a time.
#pragma once

#include "block_ops.h"
#include "ptx.cuh"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

// act(z), with a relative error of 2^-20 at most, beside what rounding the argument x of
// an exponential costs: 2^-24 |x| per rounding. Results below 2^-119 in magnitude, where
// the exponential leaves fp32's range, may come out as zero. z = -inf gives 0 for GELU by
// erf and, as the formulas do, NaN for the other two.
//
// kFull is for fp32 outputs, which show those roundings: expf, and GELU by erf with its
// exponent z^2 / 2 in two parts. A 16-bit output rounds them away (its half step is 2^-11
// or 2^-9, and |x| < 88 wherever the result counts): there the exponentials are ex2.approx
// of a rounded product.
template <bool kFull>
__device__ __forceinline__ float act_exp(float x) {
  return kFull ? expf(x) : __expf(x);
}

template <bool kFull>
__device__ __forceinline__ float apply_act(float z, int act) {
  switch (act) {
    case QKV_CTE_ACT_GELU_TANH: {
      // 0.5 z (1 + tanh u) = z / (1 + exp(-2 u)), u = sqrt(2/pi) (z + 0.044715 z^3)
      const float u2 = -1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.0f);
      return __fdividef(z, 1.0f + act_exp<kFull>(u2));
    }
    case QKV_CTE_ACT_GELU_ERF: {
      // 0.5 z (1 + erf(z / sqrt 2)) = max(z, 0) - |z| Q(|z|), Q(a) = erfc(a / sqrt 2) / 2 =
      // exp(-a^2 / 2) R(a). R is smooth and falls slowly; the polynomial of degree 8 in
      // t = 1 / (1 + 0.3 a) below was fitted to it over [0, 14.5] for the smallest largest
      // relative error (reweighted least squares), which is 2^-22.5. (A polynomial
      // fitted to erfc's absolute error, at 1.5e-7, was off by 1e-2 of the result at z = -8;
      // the library's erfcf took 1.6 times the MMAs' time at K = 5120.) Beyond 14.5 the
      // correction is 0 in fp32.
      const float a = fminf(fabsf(z), 14.5f);
      const float den = fmaf(0.3f, a, 1.0f);
      float t = __fdividef(1.0f, den);
      if (kFull) t = fmaf(t, fmaf(-den, t, 1.0f), t);  // one Newton step: R takes up to 2.7 times t's error
      float r = fmaf(t, 0.035423815f, -0.15615875f);
      r = fmaf(t, r, 0.20455723f);
      r = fmaf(t, r, -0.052034378f);
      r = fmaf(t, r, 0.12769194f);
      r = fmaf(t, r, 0.1001759f);
      r = fmaf(t, r, 0.120712146f);
      r = fmaf(t, r, 0.119632006f) * t;
      const float sq = a * a;
      float e;
      if (kFull) {  // exp(-(sq + low) / 2), low the square's rounding
        e = expf(-0.5f * sq);
        e = fmaf(e, -0.5f * fmaf(a, a, -sq), e);
      } else {
        e = __expf(-0.5f * sq);
      }
      return (z < 0.0f ? 0.0f : z) - a * (r * e);
    }
    case QKV_CTE_ACT_SILU: return __fdividef(z, 1.0f + act_exp<kFull>(-z));
    default: return z;
  }
}

// Below, kF32: the output and the residual are fp32, else of the 16-bit type e.dtype.
template <bool kF32>
__device__ __forceinline__ float load_any(const void* p, long long i, int dtype) {
  if (kF32) return static_cast<const float*>(p)[i];
  return dtype == QKV_CTE_DTYPE_BF16 ? to_f32(static_cast<const __nv_bfloat16*>(p)[i])
                                     : to_f32(static_cast<const __half*>(p)[i]);
}

template <bool kF32>
__device__ __forceinline__ void store_any(void* p, long long i, int dtype, float v) {
  if (kF32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == QKV_CTE_DTYPE_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v);
  else
    static_cast<__half*>(p)[i] = from_f32<__half>(v);
}

// 32-byte global load. Not the read-only path: the residual may be the output itself.
__device__ __forceinline__ void ld_global_v8_b32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// 16 residual elements of a row as raw words (8 for 2-byte types, 16 for fp32).
template <bool kF32>
__device__ __forceinline__ void load_residual16(const LinearEpilogue& e, long long row, int col0, uint32_t* r) {
  if constexpr (kF32) {
    const float* p = static_cast<const float*>(e.residual) + row * e.ldr + col0;
    ld_global_v8_b32(p, r);
    ld_global_v8_b32(p + 8, r + 8);
  } else {
    ld_global_v8_b32(static_cast<const uint16_t*>(e.residual) + row * e.ldr + col0, r);
  }
}

__device__ __forceinline__ float2 unpack2(uint32_t w, int dtype) {
  return dtype == QKV_CTE_DTYPE_BF16 ? unpack_pair<__nv_bfloat16>(w) : unpack_pair<__half>(w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, int dtype) {
  const float2 v = make_float2(lo, hi);
  return dtype == QKV_CTE_DTYPE_BF16 ? pack_pair<__nv_bfloat16>(v) : pack_pair<__half>(v);
}

template <int kAct, bool kF32>
__device__ __forceinline__ void activate16(float* v) {
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = apply_act<kF32>(v[j], kAct);
}

// The 16 columns at col0, whole and 32-byte aligned: v = acc * ascale (* col) + bias,
// activation, gate, the residual's raw words r, one rounding, 32-byte stores. col, bias
// and gate are the columns' values in shared memory (16-byte aligned; read by every lane
// alike), or null.
template <bool kF32>
__device__ __forceinline__ void finish16(const LinearEpilogue& e, long long row, int col0, const uint32_t* acc,
                                         float ascale, const float* col, const float* bias, const float* gate,
                                         const uint32_t* r, uint64_t pol) {
  float v[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float4 c = make_float4(ascale, ascale, ascale, ascale), b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (col != nullptr) {
      c = reinterpret_cast<const float4*>(col)[q];
      c = make_float4(c.x * ascale, c.y * ascale, c.z * ascale, c.w * ascale);
    }
    if (bias != nullptr) b = reinterpret_cast<const float4*>(bias)[q];
    v[4 * q + 0] = fmaf(__uint_as_float(acc[4 * q + 0]), c.x, b.x);
    v[4 * q + 1] = fmaf(__uint_as_float(acc[4 * q + 1]), c.y, b.y);
    v[4 * q + 2] = fmaf(__uint_as_float(acc[4 * q + 2]), c.z, b.z);
    v[4 * q + 3] = fmaf(__uint_as_float(acc[4 * q + 3]), c.w, b.w);
  }
  switch (e.act) {  // one uniform branch for the 16 columns
    case QKV_CTE_ACT_GELU_TANH: activate16<QKV_CTE_ACT_GELU_TANH, kF32>(v); break;
    case QKV_CTE_ACT_GELU_ERF: activate16<QKV_CTE_ACT_GELU_ERF, kF32>(v); break;
    case QKV_CTE_ACT_SILU: activate16<QKV_CTE_ACT_SILU, kF32>(v); break;
    default: break;
  }
  if (gate != nullptr) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 p = reinterpret_cast<const float4*>(gate)[q];
      v[4 * q + 0] *= p.x;
      v[4 * q + 1] *= p.y;
      v[4 * q + 2] *= p.z;
      v[4 * q + 3] *= p.w;
    }
  }
  if constexpr (kF32) {
    if (e.residual != nullptr) {
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(r[j]);
    }
    float* dst = static_cast<float*>(e.out) + row * e.ldo + col0;
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(v[j]);
    st_global_v8_b32_hint(dst, w, pol);
    st_global_v8_b32_hint(dst + 8, w + 8, pol);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float lo = v[2 * j], hi = v[2 * j + 1];
      if (e.residual != nullptr) {
        const float2 q = unpack2(r[j], e.dtype);
        lo += q.x;
        hi += q.y;
      }
      w[j] = pack2(lo, hi, e.dtype);
    }
    st_global_v8_b32_hint(static_cast<uint16_t*>(e.out) + row * e.ldo + col0, w, pol);
  }
}

// One element, any alignment: ragged chunks.
template <bool kF32>
__device__ __forceinline__ void finish_one(const LinearEpilogue& e, long long row, int c, float acc, float scale,
                                           float bias, float gate) {
  float v = apply_act<kF32>(fmaf(acc, scale, bias), e.act);
  if (e.gate != nullptr) v *= gate;
  if (e.residual != nullptr) v += load_any<kF32>(e.residual, row * e.ldr + c, e.dtype);
  store_any<kF32>(e.out, row * e.ldo + c, e.dtype, v);
}

}  // namespace qkvcte

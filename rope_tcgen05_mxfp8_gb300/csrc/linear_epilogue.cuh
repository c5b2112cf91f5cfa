// The product's epilogue: O = residual + gate * act(z), z = acc * scale + bias, on 16
// columns of one row at a time.
#pragma once

#include "block_ops.h"
#include "ptx.cuh"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

// act(z). The exponentials are ex2.approx of a rounded product: their relative error is
// about 2^-22 plus 2^-24 |argument|, and z / (1 + e) inherits it only in so far as e
// counts beside 1, so act is within 2^-20 |z| for any argument that does not vanish.
// e = inf gives the limit -0.
__device__ __forceinline__ float apply_act(float z, int act) {
  switch (act) {
    case QKV_CTE_ACT_GELU_TANH: {
      // 0.5 z (1 + tanh u) = z / (1 + exp(-2 u)), u = sqrt(2/pi) (z + 0.044715 z^3)
      const float u2 = -1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.0f);
      return __fdividef(z, 1.0f + __expf(u2));
    }
    case QKV_CTE_ACT_GELU_ERF: {
      // 0.5 z (1 + erf(z / sqrt 2)) = max(z, 0) - 0.5 |z| erfc(|z| / sqrt 2), with formula
      // 7.1.26 of Abramowitz and Stegun for erfc(x): t (a1 + t (a2 + ...)) exp(-x^2),
      // t = 1 / (1 + p x), off by 1.5e-7 at most (the library's erfcf took 1.6 times the
      // MMAs' time at K = 5120). Beyond |z| = 100 the correction is 0 in fp32.
      const float az = fminf(fabsf(z), 100.0f);
      const float x = 0.70710678118654752f * az;
      const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
      const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f),
                                  0.254829592f);
      return (z < 0.0f ? 0.0f : z) - 0.5f * az * poly * __expf(-x * x);
    }
    case QKV_CTE_ACT_SILU: return __fdividef(z, 1.0f + __expf(-z));
    default: return z;
  }
}

__device__ __forceinline__ float load_any(const void* p, long long i, int dtype) {
  switch (dtype) {
    case QKV_CTE_DTYPE_BF16: return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
    case QKV_CTE_DTYPE_FP16: return to_f32(static_cast<const __half*>(p)[i]);
    default: return static_cast<const float*>(p)[i];
  }
}

__device__ __forceinline__ void store_any(void* p, long long i, int dtype, float v) {
  switch (dtype) {
    case QKV_CTE_DTYPE_BF16: static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v); break;
    case QKV_CTE_DTYPE_FP16: static_cast<__half*>(p)[i] = from_f32<__half>(v); break;
    default: static_cast<float*>(p)[i] = v;
  }
}

// 32-byte global load. Not the read-only path: the residual may be the output itself.
__device__ __forceinline__ void ld_global_v8_b32(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// 16 residual elements of a row as raw words (8 for 2-byte types, 16 for fp32).
__device__ __forceinline__ void load_residual16(const LinearEpilogue& e, long long row, int col0, uint32_t* r) {
  if (e.dtype == QKV_CTE_DTYPE_FP32) {
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

// The 16 columns at col0, whole and 32-byte aligned: v = acc * ascale (* col) + bias,
// activation, gate, the residual's raw words r, one rounding, 32-byte stores. col, bias
// and gate are the columns' values in shared memory (16-byte aligned; read by every lane
// alike), or null.
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
    case QKV_CTE_ACT_GELU_TANH:
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = apply_act(v[j], QKV_CTE_ACT_GELU_TANH);
      break;
    case QKV_CTE_ACT_GELU_ERF:
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = apply_act(v[j], QKV_CTE_ACT_GELU_ERF);
      break;
    case QKV_CTE_ACT_SILU:
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = apply_act(v[j], QKV_CTE_ACT_SILU);
      break;
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
  if (e.dtype == QKV_CTE_DTYPE_FP32) {
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
    return;
  }
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

// One element, any alignment: ragged chunks.
__device__ __forceinline__ void finish_one(const LinearEpilogue& e, long long row, int c, float acc, float scale,
                                           float bias, float gate) {
  float v = apply_act(fmaf(acc, scale, bias), e.act);
  if (e.gate != nullptr) v *= gate;
  if (e.residual != nullptr) v += load_any(e.residual, row * e.ldr + c, e.dtype);
  store_any(e.out, row * e.ldo + c, e.dtype, v);
}

}  // namespace qkvcte

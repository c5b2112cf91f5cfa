// Rotary positions with several axes (time, height, width, ...): cos/sin tables, and the
// rotation of a strided tensor.
//
// Pair p of a head's d/2 pairs belongs to one axis; its angle is
//   position[axis(p)] * theta^(-e(p)),   y_lo = x_lo c - x_hi s,   y_hi = x_hi c + x_lo s
// with lanes (p, p + d/2) (rotate-half) or (2p, 2p + 1) (interleaved).
//
// Angles. A position turns by pos * theta^-e / (2 pi) turns, of which only the fraction
// counts. The step per position is kept as a 64-bit binary fraction of a turn (computed
// once on the host), so pos * step modulo 2^64 drops the whole turns exactly: no large
// angle is ever formed and a position of a million is as accurate as a small one (the
// step's own error, a few 2^-53 relative, grows with the position as it does for a
// product in 64-bit floating point). The nearest quarter turn comes off in integers as
// well; the rest, at most an eighth of a turn, is converted to fp32 (relative error
// 2^-24) for sincospif, and the quarter selects and negates. The device's 64-bit
// floating point, of which GB300 has little, is not used.
//
// Both kernels are bound by memory. A thread owns a few pairs of one token and computes
// their cos and sin once for all the heads it walks.
#include <algorithm>

#include "block_ops.h"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kHeadsPerThread = 8;  // heads a thread walks with one set of cos and sin

// cos and sin of pos * step turns (step: a binary fraction of a turn).
__device__ __forceinline__ void turn(int pos, unsigned long long step, float& c, float& s) {
  const unsigned long long u = static_cast<unsigned long long>(static_cast<long long>(pos)) * step;
  const unsigned long long q = (u + (1ull << 61)) >> 62;  // nearest quarter turn (0..3)
  const long long r = static_cast<long long>(u - (q << 62));
  float sn, cs;
  sincospif(static_cast<float>(r) * 0x1p-63f, &sn, &cs);  // 2 * (r / 2^64) half turns
  c = (q & 1) ? sn : cs;
  s = (q & 1) ? cs : sn;
  if (q == 1 || q == 2) c = -c;
  if (q >= 2) s = -s;
}

// The position of row s of batch b on every axis; false for a row behind its grid's end.
__device__ __forceinline__ bool row_position(const RopeArgs& a, int b, int s, int* pos) {
  if (a.grids == nullptr) {
    const int* p = a.positions + b * a.pos_batch_stride + static_cast<long long>(s) * a.n_axes;
#pragma unroll
    for (int i = 0; i < kRopeMaxAxes; ++i) pos[i] = i < a.n_axes ? p[i] : 0;
    return true;
  }
  const int* g = a.grids + static_cast<long long>(b) * a.n_axes;
  int left = s;
  bool live = true;
#pragma unroll
  for (int i = kRopeMaxAxes - 1; i >= 0; --i) {
    pos[i] = 0;
    if (i < a.n_axes) {
      const int size = g[i];
      live = live && size > 0;
      const int n = size > 0 ? size : 1;
      pos[i] = left % n;
      left /= n;
    }
  }
  return live && left == 0;  // s < the product of the sizes
}

__device__ __forceinline__ int pair_axis_position(const RopeArgs& a, int pair, const int* pos) {
  int v = pos[0];
#pragma unroll
  for (int i = 1; i < kRopeMaxAxes; ++i)
    if (i < a.n_axes && pair >= a.first_pair[i]) v = pos[i];
  return v;
}

// PV pairs per thread. T[PV] vectors at lo and at lo + d/2 (rotate-half), or 2 PV
// elements at 2 lo (interleaved).
template <typename T, int PV, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_apply_kernel(const __grid_constant__ RopeArgs a) {
  const int half = a.d >> 1;
  const int per_row = half / PV;
  const long long idx = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long row = idx / per_row;
  if (row >= static_cast<long long>(a.batch) * a.seq) return;
  const int p0 = static_cast<int>(idx - row * per_row) * PV;
  const int b = static_cast<int>(row / a.seq);
  const int s = static_cast<int>(row - static_cast<long long>(b) * a.seq);
  int pos[kRopeMaxAxes];
  const bool live = row_position(a, b, s, pos);
  const T* x = static_cast<const T*>(a.x) + b * a.xb + s * a.xs;
  T* y = static_cast<T*>(a.y) + b * a.yb + s * a.ys;
  if (!live && x == y) return;
  float cs[PV], sn[PV];
#pragma unroll
  for (int j = 0; j < PV; ++j) {
    turn(pair_axis_position(a, p0 + j, pos), a.step[p0 + j], cs[j], sn[j]);
    if (a.inverse) sn[j] = -sn[j];
  }
  const int h1 = min(a.heads, static_cast<int>(blockIdx.y + 1) * kHeadsPerThread);
  const int off0 = kHalf ? p0 : 2 * p0;
  const int off1 = kHalf ? p0 + half : 2 * p0 + PV;
#pragma unroll 4
  for (int h = blockIdx.y * kHeadsPerThread; h < h1; ++h) {
    const Vec<T, PV> v0 = ld_once<T, PV>(x + h * a.xh + off0);
    const Vec<T, PV> v1 = ld_once<T, PV>(x + h * a.xh + off1);
    Vec<T, PV> o0 = v0, o1 = v1;
    if (live) {
#pragma unroll
      for (int j = 0; j < PV; ++j) {
        // interleaved: element 2j of the 2 PV (v0 then v1) and its neighbour
        const float lo = to_f32(kHalf ? v0.v[j] : (2 * j < PV ? v0.v[2 * j % PV] : v1.v[2 * j % PV]));
        const float hi = to_f32(kHalf ? v1.v[j] : (2 * j + 1 < PV ? v0.v[(2 * j + 1) % PV] : v1.v[(2 * j + 1) % PV]));
        const T ylo = from_f32<T>(lo * cs[j] - hi * sn[j]);
        const T yhi = from_f32<T>(hi * cs[j] + lo * sn[j]);
        if (kHalf) {
          o0.v[j] = ylo;
          o1.v[j] = yhi;
        } else {
          if (2 * j < PV) o0.v[2 * j % PV] = ylo; else o1.v[2 * j % PV] = ylo;
          if (2 * j + 1 < PV) o0.v[(2 * j + 1) % PV] = yhi; else o1.v[(2 * j + 1) % PV] = yhi;
        }
      }
    }
    st_vec(y + h * a.yh + off0, o0);
    st_vec(y + h * a.yh + off1, o1);
  }
}

// Tables: fp32 [batch * seq, d], each pair's value at both of its lanes.
template <int PV, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_tables_kernel(const __grid_constant__ RopeArgs a, float* cos_t,
                                                                   float* sin_t) {
  const int half = a.d >> 1;
  const int per_row = half / PV;
  const long long idx = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long row = idx / per_row;
  if (row >= static_cast<long long>(a.batch) * a.seq) return;
  const int p0 = static_cast<int>(idx - row * per_row) * PV;
  const int b = static_cast<int>(row / a.seq);
  int pos[kRopeMaxAxes];
  const bool live = row_position(a, b, static_cast<int>(row - static_cast<long long>(b) * a.seq), pos);
  Vec<float, PV> c, s;
#pragma unroll
  for (int j = 0; j < PV; ++j) {
    c.v[j] = 1.0f;
    s.v[j] = 0.0f;
    if (live) turn(pair_axis_position(a, p0 + j, pos), a.step[p0 + j], c.v[j], s.v[j]);
  }
  float* cr = cos_t + row * a.d;
  float* sr = sin_t + row * a.d;
  if constexpr (kHalf) {
    st_vec(cr + p0, c);
    st_vec(cr + p0 + half, c);
    st_vec(sr + p0, s);
    st_vec(sr + p0 + half, s);
  } else {
#pragma unroll
    for (int j = 0; j < PV; ++j) {
      st_vec(cr + 2 * (p0 + j), Vec<float, 2>{{c.v[j], c.v[j]}});
      st_vec(sr + 2 * (p0 + j), Vec<float, 2>{{s.v[j], s.v[j]}});
    }
  }
}

template <typename T, int PV, bool kHalf>
cudaError_t apply_go(const RopeArgs& a, cudaStream_t s) {
  const long long threads = static_cast<long long>(a.batch) * a.seq * ((a.d >> 1) / PV);
  const long long blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  const dim3 grid(static_cast<unsigned>(blocks), (a.heads + kHeadsPerThread - 1) / kHeadsPerThread);
  rope_apply_kernel<T, PV, kHalf><<<grid, kRopeThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool kHalf>
cudaError_t apply_t(const RopeArgs& a, cudaStream_t s) {
  // the widest access that divides a head's pairs and that pointers and strides allow
  int pv = 16 / static_cast<int>(sizeof(T));
  const uintptr_t where = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
  const long long strides = a.xb | a.xs | a.xh | a.yb | a.ys | a.yh;
  while (pv > 1 && ((a.d >> 1) % pv != 0 || where % (pv * sizeof(T)) != 0 || strides % pv != 0)) pv >>= 1;
  switch (pv) {
    case 8:
      if constexpr (sizeof(T) == 2) return apply_go<T, 8, kHalf>(a, s);
    case 4: return apply_go<T, 4, kHalf>(a, s);
    case 2: return apply_go<T, 2, kHalf>(a, s);
    default: return apply_go<T, 1, kHalf>(a, s);
  }
}

template <int PV, bool kHalf>
cudaError_t tables_go(const RopeArgs& a, float* cos_t, float* sin_t, cudaStream_t s) {
  const long long threads = static_cast<long long>(a.batch) * a.seq * ((a.d >> 1) / PV);
  rope_tables_kernel<PV, kHalf>
      <<<static_cast<unsigned>((threads + kRopeThreads - 1) / kRopeThreads), kRopeThreads, 0, s>>>(a, cos_t, sin_t);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_apply(const RopeArgs& a, int dtype, bool rotate_half, cudaStream_t s) {
  if (static_cast<long long>(a.batch) * a.seq * a.heads == 0) return cudaSuccess;
  switch (dtype) {
    case QKV_CTE_DTYPE_BF16:
      return rotate_half ? apply_t<__nv_bfloat16, true>(a, s) : apply_t<__nv_bfloat16, false>(a, s);
    case QKV_CTE_DTYPE_FP16: return rotate_half ? apply_t<__half, true>(a, s) : apply_t<__half, false>(a, s);
    default: return rotate_half ? apply_t<float, true>(a, s) : apply_t<float, false>(a, s);
  }
}

cudaError_t launch_rope_tables(const RopeArgs& a, float* cos_t, float* sin_t, bool rotate_half, cudaStream_t s) {
  if (static_cast<long long>(a.batch) * a.seq == 0) return cudaSuccess;
  const int half = a.d >> 1;
  const uintptr_t where = reinterpret_cast<uintptr_t>(cos_t) | reinterpret_cast<uintptr_t>(sin_t);
  if (rotate_half) {
    if (half % 4 == 0 && where % 16 == 0) return tables_go<4, true>(a, cos_t, sin_t, s);
    if (half % 2 == 0 && where % 8 == 0) return tables_go<2, true>(a, cos_t, sin_t, s);
    return tables_go<1, true>(a, cos_t, sin_t, s);
  }
  if (half % 2 == 0) return tables_go<2, false>(a, cos_t, sin_t, s);
  return tables_go<1, false>(a, cos_t, sin_t, s);
}

}  // namespace qkvcte

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
// The rotation is bound by memory: a thread owns a few pairs of one token and computes
// their cos and sin once for all the heads it walks. 32760 x 40 heads of 128 lanes in bf16,
// 16-byte accesses: 104 us rotate-half and 102 interleaved in a captured graph (floor 99).
// Pair counts that narrow the accesses cost: heads of 132 lanes (4 and 8 bytes) 135 and 126 us
// (floor 102), of 126 lanes (2 and 4 bytes) 231 and 167 (floor 97). The tables are bound by
// their 100 instructions per angle: 32760 x 128 takes 10.6 us from positions and 11.4 from a
// grid, interleaved 18.0 and 19.4 (floor 4.9).
#include <algorithm>

#include "block_ops.h"
#include "fp32x2.cuh"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

namespace {

constexpr int kRopeThreads = 256;
// Heads a thread turns with one set of cos and sin, all of them requested before cos and
// sin are computed. 32760 x 40 heads of 128 in bf16: 107 us with 8 heads; 121 with 8
// requested 4 at a time, 125 with 20, 135 with 40.
constexpr int kHeadsPerThread = 8;

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

// PV pairs per thread: vectors of PV elements at lane p0 and at p0 + d/2 (rotate-half), or
// one of 2 PV elements at 2 p0 (interleaved). cos and sin are computed while the heads' loads are in flight.
template <typename T, int PV>
struct HalfPairs {
  using V = Vec<T, PV>;
  V lo, hi;
  __device__ __forceinline__ void load(const T* x, int p0, int half) {
    lo = ld_once<T, PV>(x + p0);
    hi = ld_once<T, PV>(x + p0 + half);
  }
  __device__ __forceinline__ void store(T* y, int p0, int half) const {
    st_vec(y + p0, lo);
    st_vec(y + p0 + half, hi);
  }
  __device__ __forceinline__ void rotate(const float* c, const float* s) {
    if constexpr (PV == 1) {
      const float a = lo.one(), b = hi.one();
      lo.set_one(a * c[0] - b * s[0]);
      hi.set_one(b * c[0] + a * s[0]);
    } else {
#pragma unroll
      for (int j = 0; j < PV / 2; ++j) {
        const float2 a = lo.pair(j), b = hi.pair(j);
        const float2 cc = make_float2(c[2 * j], c[2 * j + 1]), ss = make_float2(s[2 * j], s[2 * j + 1]);
        lo.set_pair(j, ffma2(a, cc, fmul2(b, make_float2(-ss.x, -ss.y))));
        hi.set_pair(j, ffma2(b, cc, fmul2(a, ss)));
      }
    }
  }
};

template <typename T, int PV>
struct NeighbourPairs {
  using V = Vec<T, 2 * PV>;
  V v;
  __device__ __forceinline__ void load(const T* x, int p0, int) { v = ld_once<T, 2 * PV>(x + 2 * p0); }
  __device__ __forceinline__ void store(T* y, int p0, int) const { st_vec(y + 2 * p0, v); }
  __device__ __forceinline__ void rotate(const float* c, const float* s) {
#pragma unroll
    for (int j = 0; j < PV; ++j) {
      const float2 a = v.pair(j);
      v.set_pair(j, make_float2(a.x * c[j] - a.y * s[j], a.y * c[j] + a.x * s[j]));
    }
  }
};

// Neighbouring lanes at an address that keeps no pair together (2-byte aligned only).
template <typename T>
struct ScatteredPair {
  Vec<T, 1> lo, hi;
  __device__ __forceinline__ void load(const T* x, int p0, int) {
    lo = ld_once<T, 1>(x + 2 * p0);
    hi = ld_once<T, 1>(x + 2 * p0 + 1);
  }
  __device__ __forceinline__ void store(T* y, int p0, int) const {
    st_vec(y + 2 * p0, lo);
    st_vec(y + 2 * p0 + 1, hi);
  }
  __device__ __forceinline__ void rotate(const float* c, const float* s) {
    const float a = lo.one(), b = hi.one();
    lo.set_one(a * c[0] - b * s[0]);
    hi.set_one(b * c[0] + a * s[0]);
  }
};

template <typename T, int PV, typename Pairs>
__global__ void __launch_bounds__(kRopeThreads) rope_apply_kernel(const __grid_constant__ RopeArgs a) {
  const int half = a.d >> 1;
  const int per_row = half / PV;
  const long long idx = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const long long row = idx / per_row;
  if (row >= static_cast<long long>(a.batch) * a.seq) return;
  const int p0 = static_cast<int>(idx - row * per_row) * PV;
  const int b = static_cast<int>(row / a.seq);
  const int s = static_cast<int>(row - static_cast<long long>(b) * a.seq);
  const int h0 = blockIdx.y * kHeadsPerThread;
  const T* x = static_cast<const T*>(a.x) + b * a.xb + s * a.xs + h0 * a.xh;
  T* y = static_cast<T*>(a.y) + b * a.yb + s * a.ys + h0 * a.yh;
  const int n = min(a.heads - h0, kHeadsPerThread);
  Pairs v[kHeadsPerThread];
#pragma unroll
  for (int k = 0; k < kHeadsPerThread; ++k)
    if (k < n) v[k].load(x + k * a.xh, p0, half);
  int pos[kRopeMaxAxes];
  const bool live = row_position(a, b, s, pos);
  if (!live && a.x == a.y) return;  // padding in place
  float cs[PV], sn[PV];
#pragma unroll
  for (int j = 0; j < PV; ++j) {
    turn(pair_axis_position(a, p0 + j, pos), a.step[p0 + j], cs[j], sn[j]);
    if (a.inverse) sn[j] = -sn[j];
  }
#pragma unroll
  for (int k = 0; k < kHeadsPerThread; ++k) {
    if (k < n) {
      if (live) v[k].rotate(cs, sn);  // padding rows keep their values, whatever they are
      v[k].store(y + k * a.yh, p0, half);
    }
  }
}

// The same PV values at two places of a table row.
template <int PV>
__device__ __forceinline__ void store_table(float* p, float* q, const float* v) {
  Vec<float, PV> o;
  if constexpr (PV == 1) {
    o.set_one(v[0]);
  } else {
#pragma unroll
    for (int j = 0; j < PV / 2; ++j) o.set_pair(j, make_float2(v[2 * j], v[2 * j + 1]));
  }
  st_vec(p, o);
  st_vec(q, o);
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
  float c[PV], s[PV];
#pragma unroll
  for (int j = 0; j < PV; ++j) {
    c[j] = 1.0f;
    s[j] = 0.0f;
    if (live) turn(pair_axis_position(a, p0 + j, pos), a.step[p0 + j], c[j], s[j]);
  }
  float* cr = cos_t + row * a.d;
  float* sr = sin_t + row * a.d;
  if constexpr (kHalf) {
    store_table<PV>(cr + p0, cr + p0 + half, c);
    store_table<PV>(sr + p0, sr + p0 + half, s);
  } else {
#pragma unroll
    for (int j = 0; j < PV; ++j) {
      reinterpret_cast<float2*>(cr)[p0 + j] = make_float2(c[j], c[j]);
      reinterpret_cast<float2*>(sr)[p0 + j] = make_float2(s[j], s[j]);
    }
  }
}

template <typename T, int PV, typename Pairs>
cudaError_t apply_go(const RopeArgs& a, cudaStream_t s) {
  const long long threads = static_cast<long long>(a.batch) * a.seq * ((a.d >> 1) / PV);
  const long long blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  const dim3 grid(static_cast<unsigned>(blocks), (a.heads + kHeadsPerThread - 1) / kHeadsPerThread);
  rope_apply_kernel<T, PV, Pairs><<<grid, kRopeThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// The widest access that divides a head's pairs and that pointers and strides allow.
template <typename T>
cudaError_t apply_t(const RopeArgs& a, bool rotate_half, cudaStream_t s) {
  const int half = a.d >> 1;
  const uintptr_t where = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y);
  const long long strides = a.xb | a.xs | a.xh | a.yb | a.ys | a.yh;
  int n = 16 / static_cast<int>(sizeof(T));  // elements per access
  while (n > 1 && ((rotate_half ? half % n : a.d % n) != 0 || where % (n * sizeof(T)) != 0 || strides % n != 0)) n >>= 1;
  if (rotate_half) {
    switch (n) {
      case 8:
        if constexpr (sizeof(T) == 2) return apply_go<T, 8, HalfPairs<T, 8>>(a, s);
      case 4: return apply_go<T, 4, HalfPairs<T, 4>>(a, s);
      case 2: return apply_go<T, 2, HalfPairs<T, 2>>(a, s);
      default: return apply_go<T, 1, HalfPairs<T, 1>>(a, s);
    }
  }
  switch (n) {
    case 8:
      if constexpr (sizeof(T) == 2) return apply_go<T, 4, NeighbourPairs<T, 4>>(a, s);
    case 4: return apply_go<T, 2, NeighbourPairs<T, 2>>(a, s);
    case 2: return apply_go<T, 1, NeighbourPairs<T, 1>>(a, s);
    default: return apply_go<T, 1, ScatteredPair<T>>(a, s);
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
    case QKV_CTE_DTYPE_BF16: return apply_t<__nv_bfloat16>(a, rotate_half, s);
    case QKV_CTE_DTYPE_FP16: return apply_t<__half>(a, rotate_half, s);
    default: return apply_t<float>(a, rotate_half, s);
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

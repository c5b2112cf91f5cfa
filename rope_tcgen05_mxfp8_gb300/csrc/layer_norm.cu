// Layer norm over the last dimension, forward and backward.
//
//   mu = mean(x), var = mean((x - mu)^2), r = 1 / sqrt(var + eps), xh = (x - mu) r
//   y  = xh * w + b
//   g  = dy * w,  dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Both passes are bound by memory (2 and 3 times the tensor). A row belongs to one group
// of threads (a warp for short rows, a block for long ones) and is read once; the
// variance is taken about the mean in a second sweep over the registers, never as a
// difference of large sums. Rows come through a ring in shared memory that each thread
// fills for itself with 16-byte asynchronous copies, two or three rows ahead, so that loads
// stay in flight across the reductions (rows off 16-byte boundaries: the group copies the
// pieces that cover them); parameters stay in registers over all the rows of a block. The
// backward pass keeps its column sums dw and db in the registers of the same threads,
// adds those of a cluster of four blocks on chip, and a second kernel adds the clusters'
// in a fixed order (no atomics: the result does not depend on the schedule).
// Sums, statistics and gradients are fp32; outputs are rounded once.
//
// Arithmetic counts: a first form that converted each element in each sweep, read the
// parameters from L1 and prefetched one row into registers ran 24 instructions per
// element and took 204 us for 32760 x 5120 in bf16, twice the floor. Elements are
// converted once, worked on in pairs (fma.rn.f32x2 and so on) and kept as x - mu: 101 us
// (6.6 TB/s, 98 % of the measured copy rate). Backward, 4096 x 5120: 33 us with the join
// of the column sums (3.8 TB/s); 32760 x 5120: 173 us (5.8 TB/s). Figures here are bf16 rows
// in a captured graph.
#include <algorithm>

#include "block_ops.h"
#include "fp32x2.cuh"
#include "ptx.cuh"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

namespace {

constexpr int kWarpRows = 4;  // rows (warps) per block of the warp-per-row form

constexpr int kGradCluster = 4;  // blocks whose column sums are joined on chip

// Sums of N values over the group of threads that holds a row: a warp (blockDim.x ==
// 32, no barrier) or the whole block of at most 4 * kQuads warps. `slot` alternates
// between consecutive calls: a thread writes a slot again only after the barrier of the
// call in between, which every reader of the slot has reached. The entries of absent
// warps must hold zeros (clear_sums). Per thread: its terms, five levels in the warp,
// then kQuads additions in four lanes and two more.
template <int N, int kQuads>
struct GroupSums {
  float4 v[2][N][kQuads];
};

template <int N, int kQuads>
__device__ __forceinline__ void clear_sums(GroupSums<N, kQuads>& red) {
  if (blockDim.x == 32) return;
  float* p = reinterpret_cast<float*>(&red);
  for (int i = threadIdx.x; i < 2 * N * 4 * kQuads; i += blockDim.x) p[i] = 0.0f;
  __syncthreads();
}

template <int N, int kQuads>
__device__ __forceinline__ void group_sum(float* v, GroupSums<N, kQuads>& red, int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (blockDim.x == 32) return;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) reinterpret_cast<float*>(red.v[slot][k])[threadIdx.x >> 5] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    float4 t = red.v[slot][k][0];
#pragma unroll
    for (int q = 1; q < kQuads; ++q) {
      const float4 r = red.v[slot][k][q];
      t = make_float4(t.x + r.x, t.y + r.y, t.z + r.z, t.w + r.w);
    }
    v[k] = (t.x + t.y) + (t.z + t.w);
  }
}

// What a thread computes on: pairs where an access holds several elements, else single
// elements.
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) { return ffma2(a, b, c); }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return fmul2(a, b); }
__device__ __forceinline__ float2 vadd(float2 a, float2 b) { return fadd2(a, b); }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float hsum(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float hsum(float a) { return a; }

template <int VEC>
struct Lanes {
  static_assert(VEC % 2 == 0, "pairs");
  using F = float2;
  static constexpr int N = VEC / 2;
  static __device__ __forceinline__ F all(float x) { return make_float2(x, x); }
  template <typename V>
  static __device__ __forceinline__ F get(const V& v, int j) {
    return v.pair(j);
  }
  template <typename V>
  static __device__ __forceinline__ void put(V& v, int j, F x) {
    v.set_pair(j, x);
  }
};
template <>
struct Lanes<1> {
  using F = float;
  static constexpr int N = 1;
  static __device__ __forceinline__ F all(float x) { return x; }
  template <typename V>
  static __device__ __forceinline__ F get(const V& v, int) {
    return v.one();
  }
  template <typename V>
  static __device__ __forceinline__ void put(V& v, int, F x) {
    v.set_one(x);
  }
};

// A thread's part of a row: CH accesses of VEC elements, blockDim.x accesses apart (kFull:
// the row fills them all), and the ring of rows on their way. Whole 16-byte accesses: each
// thread copies its own and reads back what it copied, without a barrier. Single elements
// (rows off 16-byte boundaries): the group copies the 16-byte pieces that cover the row
// and each thread takes its elements out of them, so a barrier goes before and after.
// (The first and the last piece may reach past the row's ends, never past the aligned 16
// bytes that hold one of its elements.)
template <typename T, int VEC, int CH, bool kFull, int kRows>
struct RowStream {
  static constexpr bool kOwn = VEC > 1;
  static constexpr int kAhead = kRows;  // rows kept requested

  const T* next;   // kOwn: this thread's first element of the next row to request, else the row
  long long pitch; // elements to the one after
  int left;        // rows still to request
  uint32_t ring;   // shared address of the group's ring (kOwn: of this thread's first access)
  uint32_t stride; // kOwn: bytes from one of a row's accesses to the next; else from row to row
  uint32_t shift;  // !kOwn: bytes of the current row's first piece before the row
  uint32_t turn;   // !kOwn: what the shift grows by from row to row (modulo 16)

  // Shared memory of a block's ring.
  static __host__ __device__ __forceinline__ uint32_t row_bytes(int cols) {
    return (static_cast<uint32_t>(cols) * sizeof(T) + 15 + 15) / 16 * 16;  // any shift
  }
  static __host__ __device__ __forceinline__ uint32_t bytes(int cols, int threads_x, int threads_y) {
    return kAhead * (kOwn ? CH * 16u * threads_x : row_bytes(cols)) * threads_y;
  }
  static __device__ __forceinline__ bool inside(int i, int cols) {
    return kFull || static_cast<int>(i * blockDim.x + threadIdx.x) * VEC < cols;
  }
  // The group takes rows first, first + step, ... below rows.
  __device__ __forceinline__ void init(uint8_t* base, const void* p, long long ld, int cols, int first, int step,
                                       int rows) {
    next = static_cast<const T*>(p) + first * ld;
    pitch = step * ld;
    left = first < rows ? (rows - 1 - first) / step + 1 : 0;
    ring = static_cast<uint32_t>(__cvta_generic_to_shared(base));
    if constexpr (kOwn) {
      next += threadIdx.x * VEC;
      stride = 16 * blockDim.x * blockDim.y;
      ring += 16 * (threadIdx.y * blockDim.x + threadIdx.x);
    } else {
      stride = row_bytes(cols);
      ring += threadIdx.y * kAhead * stride;
      shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(next) & 15);
      turn = static_cast<uint32_t>(pitch * static_cast<long long>(sizeof(T))) & 15;
    }
  }
  // Request the next row, if there is one, into ring slot `slot`.
  __device__ __forceinline__ void request(int cols, int slot) {
    if (left > 0) {
      if constexpr (kOwn) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (inside(i, cols)) cp_async16(ring + (slot * CH + i) * stride, next + i * blockDim.x * VEC);
      } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(next);
        const uintptr_t end = at + static_cast<uintptr_t>(cols) * sizeof(T);
        uint32_t dst = ring + slot * stride + 16 * threadIdx.x;
        for (uintptr_t src = (at & ~uintptr_t(15)) + 16 * threadIdx.x; src < end; src += 16 * blockDim.x) {
          cp_async16(dst, reinterpret_cast<const void*>(src));
          dst += 16 * blockDim.x;
        }
      }
      next += pitch;
      --left;
    }
  }
  // After the wait for this thread's copies: the row is there for every thread.
  __device__ __forceinline__ void arrived() const {
    if constexpr (!kOwn) sync_group();
  }
  // Every thread has taken what it wants of the current row.
  __device__ __forceinline__ void taken() const {
    if constexpr (!kOwn) sync_group();
  }
  static __device__ __forceinline__ void sync_group() {
    if (blockDim.x == 32)
      __syncwarp();
    else
      __syncthreads();
  }
  __device__ __forceinline__ void advance() {
    if constexpr (!kOwn) shift = (shift + turn) & 15;
  }
  __device__ __forceinline__ Vec<T, VEC> take(int i, int slot) const {
    Vec<T, VEC> r;
    if constexpr (kOwn) {
      ld_shared16(ring + (slot * CH + i) * stride, r.w);
    } else {
      r.v = ld_shared_elem<T>(ring + slot * stride + shift +
                              static_cast<uint32_t>((i * blockDim.x + threadIdx.x) * sizeof(T)));
    }
    return r;
  }
};

// A thread's part of the parameters, packed (`absent` without a tensor).
template <typename P, int VEC, int CH>
struct ParamPart {
  using L = Lanes<VEC>;
  static constexpr int N = 16 / sizeof(P) < VEC ? 16 / sizeof(P) : VEC;  // per access
  static constexpr int kPer = VEC == 1 ? 1 : N / 2;                       // lanes per access
  Vec<P, N> v[CH][VEC / N];

  // The parameters of accesses first, first + 1, ...
  __device__ __forceinline__ void load(const void* p, int cols, float absent, int first = 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = ((first + i) * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
      for (int k = 0; k < VEC / N; ++k) {
        if (p != nullptr && c < cols) {
          v[i][k] = *reinterpret_cast<const Vec<P, N>*>(static_cast<const P*>(p) + c + k * N);
        } else {
#pragma unroll
          for (int j = 0; j < kPer; ++j) L::put(v[i][k], j, L::all(absent));
        }
      }
    }
  }
  __device__ __forceinline__ typename L::F get(int i, int j) const { return L::get(v[i][j / kPer], j % kPer); }
};

// Forms of the kernels: kKeep holds the parameters in registers over all rows, else they
// are read for every row; kFull rows fill every access of every thread.
template <typename T_, typename P_, int VEC_, int CH_, bool kKeep_, bool kFull_>
struct Form {
  using T = T_;
  using P = P_;
  static constexpr int VEC = VEC_, CH = CH_;
  static constexpr bool kKeep = kKeep_, kFull = kFull_;
  using L = Lanes<VEC>;
  // Rows in flight: 32760 x 5120 bf16 forward 118 us with two and 120 with three at four
  // accesses per thread, backward 182 and 175.
  using Forward = RowStream<T, VEC, CH, kFull, (VEC > 1 && CH > 4 ? 1 : (VEC > 1 && CH > 2 ? 2 : 3))>;
  using Backward = RowStream<T, VEC, CH, kFull, 3>;
};

// Backward: kept parameters and column sums leave registers for 256 threads only.
template <typename Fm>
constexpr int kGradThreads = Fm::kKeep && Fm::VEC > 1 ? 256 : 512;

template <typename Fm>
__global__ void __launch_bounds__(512) layer_norm_kernel(LayerNormArgs a) {
  using T = typename Fm::T;
  using L = typename Fm::L;
  using F = typename L::F;
  using Stream = typename Fm::Forward;
  constexpr int VEC = Fm::VEC, CH = Fm::CH, kAhead = Stream::kAhead;
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ GroupSums<1, 4> red;
  const float inv = 1.0f / static_cast<float>(a.cols);
  const int step = gridDim.x * blockDim.y;
  const int first = blockIdx.x * blockDim.y + threadIdx.y;
  Stream in;
  in.init(ring_mem, a.x, a.ldx, a.cols, first, step, static_cast<int>(a.rows));
  const int n = in.left;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    in.request(a.cols, k);
    cp_async_commit();
  }
  ParamPart<typename Fm::P, VEC, Fm::kKeep ? CH : 1> wp, bp;
  if (Fm::kKeep) {
    wp.load(a.weight, a.cols, 1.0f);
    bp.load(a.bias, a.cols, 0.0f);
  }
  clear_sums(red);
  T* out = static_cast<T*>(a.y) + first * a.ldy + threadIdx.x * VEC;
  int slot = 0;
  for (int k = 0; k < n; ++k) {
    cp_async_wait<kAhead - 1>();
    in.arrived();
    F d[CH][L::N];
    F s = L::all(0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (Stream::inside(i, a.cols)) {
        const Vec<T, VEC> v = in.take(i, slot);
#pragma unroll
        for (int j = 0; j < L::N; ++j) {
          d[i][j] = L::get(v, j);
          s = vadd(s, d[i][j]);
        }
      }
    }
    in.taken();  // the slot is free
    in.request(a.cols, slot);
    in.advance();
    cp_async_commit();
    slot = slot + 1 == kAhead ? 0 : slot + 1;
    float sum = hsum(s);
    group_sum(&sum, red, 0);
    const float mean = sum * inv;
    F ss = L::all(0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (Stream::inside(i, a.cols)) {
#pragma unroll
        for (int j = 0; j < L::N; ++j) {
          d[i][j] = vadd(d[i][j], L::all(-mean));
          ss = vfma(d[i][j], d[i][j], ss);
        }
      }
    }
    sum = hsum(ss);
    group_sum(&sum, red, 1);
    const float rstd = rsqrtf(fmaf(sum, inv, a.eps));
    if (threadIdx.x == 0) {
      const long long row = first + static_cast<long long>(k) * step;
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (Stream::inside(i, a.cols)) {
        if (!Fm::kKeep) {
          wp.load(a.weight, a.cols, 1.0f, i);
          bp.load(a.bias, a.cols, 0.0f, i);
        }
        const int k = Fm::kKeep ? i : 0;
        Vec<T, VEC> o;
#pragma unroll
        for (int j = 0; j < L::N; ++j)
          L::put(o, j, vfma(vmul(d[i][j], L::all(rstd)), wp.get(k, j), bp.get(k, j)));
        st_vec(out + i * blockDim.x * VEC, o);
      }
    }
    out += step * a.ldy;
  }
}

// Rows longer than the registers of a block: read three times (from L2 after the first),
// element by element. 2000 x 40000: 247 us (floor 47); 4000 x 9001, off 16-byte boundaries:
// 120 us (floor 21).
template <typename T, typename P>
__global__ void __launch_bounds__(1024) layer_norm_long_kernel(LayerNormArgs a) {
  __shared__ GroupSums<1, 8> red;
  clear_sums(red);
  const float inv = 1.0f / static_cast<float>(a.cols);
  const P* w = static_cast<const P*>(a.weight);
  const P* b = static_cast<const P*>(a.bias);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
    T* yr = static_cast<T*>(a.y) + row * a.ldy;
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) s += to_f32(xr[c]);
    group_sum(&s, red, 0);
    const float mean = s * inv;
    float ss = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float d = to_f32(xr[c]) - mean;
      ss = fmaf(d, d, ss);
    }
    group_sum(&ss, red, 1);
    const float rstd = rsqrtf(fmaf(ss, inv, a.eps));
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float xh = (to_f32(xr[c]) - mean) * rstd;
      yr[c] = from_f32<T>(fmaf(xh, w != nullptr ? to_f32(w[c]) : 1.0f, b != nullptr ? to_f32(b[c]) : 0.0f));
    }
  }
}

// Columns fixed to threads; a cluster's column sums leave as one row of the workspace.
// The second sweep takes the row from the ring again: keeping xh and g instead cost 64
// registers at four accesses per thread, and with them the second block on an SM.
template <typename Fm>
__global__ void __launch_bounds__(kGradThreads<Fm>) layer_norm_backward_kernel(LayerNormGradArgs a) {
  using T = typename Fm::T;
  using L = typename Fm::L;
  using F = typename L::F;
  using Stream = typename Fm::Backward;
  constexpr int VEC = Fm::VEC, CH = Fm::CH, kAhead = Stream::kAhead;
  // the ring; after the last row, [2][cols] column sums
  extern __shared__ __align__(16) uint8_t ring_mem[];
  __shared__ GroupSums<2, kGradThreads<Fm> / 128> red;
  const float inv = 1.0f / static_cast<float>(a.cols);
  const int step = gridDim.x * blockDim.y;
  const int first = blockIdx.x * blockDim.y + threadIdx.y;
  const int rows = static_cast<int>(a.rows);
  Stream xin, gin;
  xin.init(ring_mem, a.x, a.ldx, a.cols, first, step, rows);
  gin.init(ring_mem + Stream::bytes(a.cols, blockDim.x, blockDim.y), a.dy, a.lddy, a.cols, first, step, rows);
  const int n = xin.left;
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    xin.request(a.cols, k);
    gin.request(a.cols, k);
    cp_async_commit();
  }
  const float* mean_p = a.mean + first;
  const float* rstd_p = a.rstd + first;
  float mean = n > 0 ? *mean_p : 0.0f, rstd = n > 0 ? *rstd_p : 0.0f;
  ParamPart<typename Fm::P, VEC, Fm::kKeep ? CH : 1> wp;
  if (Fm::kKeep) wp.load(a.weight, a.cols, 1.0f);
  clear_sums(red);
  F dw[CH][L::N], db[CH][L::N];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < L::N; ++j) dw[i][j] = db[i][j] = L::all(0.0f);
  T* out_row = a.dx != nullptr ? static_cast<T*>(a.dx) + first * a.lddx + threadIdx.x * VEC : nullptr;
  int slot = 0;
  for (int k = 0; k < n; ++k) {
    float mean_next = 0.0f, rstd_next = 0.0f;  // requested a whole row before their use
    if (k + 1 < n) {
      mean_next = *(mean_p += step);
      rstd_next = *(rstd_p += step);
    }
    cp_async_wait<kAhead - 1>();
    xin.arrived();
    F s1 = L::all(0.0f), s2 = L::all(0.0f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (Stream::inside(i, a.cols)) {
        const Vec<T, VEC> xv = xin.take(i, slot), gv = gin.take(i, slot);
        if (!Fm::kKeep) wp.load(a.weight, a.cols, 1.0f, i);
#pragma unroll
        for (int j = 0; j < L::N; ++j) {
          const F d = L::get(gv, j);
          const F xh = vmul(vadd(L::get(xv, j), L::all(-mean)), L::all(rstd));
          const F g = vmul(d, wp.get(Fm::kKeep ? i : 0, j));
          s1 = vadd(s1, g);
          s2 = vfma(g, xh, s2);
          dw[i][j] = vfma(d, xh, dw[i][j]);
          db[i][j] = vadd(db[i][j], d);
        }
      }
    }
    if (a.dx != nullptr) {  // uniform over the grid
      float c[2] = {hsum(s1), hsum(s2)};
      group_sum(c, red, k & 1);
      // dx = r (g - c1 - xh c2) with xh = (x - mean) r
      const F c1 = L::all(-c[0] * inv), c2 = L::all(-c[1] * inv);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        if (Stream::inside(i, a.cols)) {
          const Vec<T, VEC> xv = xin.take(i, slot), gv = gin.take(i, slot);
          if (!Fm::kKeep) wp.load(a.weight, a.cols, 1.0f, i);
          Vec<T, VEC> o;
#pragma unroll
          for (int j = 0; j < L::N; ++j) {
            const F xh = vmul(vadd(L::get(xv, j), L::all(-mean)), L::all(rstd));
            const F g = vmul(L::get(gv, j), wp.get(Fm::kKeep ? i : 0, j));
            L::put(o, j, vmul(vadd(vfma(xh, c2, g), c1), L::all(rstd)));
          }
          st_vec(out_row + i * blockDim.x * VEC, o);
        }
      }
      out_row += step * a.lddx;
    }
    xin.taken();  // the slot is free
    xin.request(a.cols, slot);
    gin.request(a.cols, slot);
    xin.advance();
    gin.advance();
    cp_async_commit();
    slot = slot + 1 == kAhead ? 0 : slot + 1;
    mean = mean_next;
    rstd = rstd_next;
  }
  if (a.partial == nullptr) return;
  // The block's column sums [2][cols] to shared memory (several rows per block: the warps
  // one after the other), then the cluster's blocks added in order, each block taking a
  // share of the columns: one partial row per cluster goes to the workspace.
  float* sums = reinterpret_cast<float*>(ring_mem);
  cp_async_wait<0>();
  __syncthreads();  // no thread reads the ring any more
  for (int r = 0; r < static_cast<int>(blockDim.y); ++r) {
    if (static_cast<int>(threadIdx.y) == r) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = (i * blockDim.x + threadIdx.x) * VEC;
        if (Stream::inside(i, a.cols)) {
#pragma unroll
          for (int j = 0; j < L::N; ++j) {
            F* p = reinterpret_cast<F*>(sums + c) + j;  // cols is even where F is a pair
            *p = r == 0 ? dw[i][j] : vadd(*p, dw[i][j]);
            p = reinterpret_cast<F*>(sums + a.cols + c) + j;
            *p = r == 0 ? db[i][j] : vadd(*p, db[i][j]);
          }
        }
      }
    }
    if (blockDim.y > 1) __syncthreads();
  }
  cluster_sync();
  const uint32_t base = smem_u32(sums);
  const int threads = blockDim.x * blockDim.y;
  float* out = a.partial + static_cast<size_t>(blockIdx.x / kGradCluster) * 2 * a.cols;
  for (int c = cluster_ctarank() * threads + threadIdx.y * blockDim.x + threadIdx.x; c < 2 * a.cols;
       c += kGradCluster * threads) {
    float v[kGradCluster];
#pragma unroll
    for (int r = 0; r < kGradCluster; ++r) v[r] = ld_shared_cluster_f32(mapa_shared(base + 4 * c, r));
    float t = v[0];
#pragma unroll
    for (int r = 1; r < kGradCluster; ++r) t += v[r];
    out[c] = t;
  }
  cluster_sync();  // no block leaves while another reads its sums
}

// Rows longer than the registers, element by element: 2000 x 20000 205 us (floor 35; the
// ring's form takes 64 for 2000 x 16384, floor 29), 2000 x 12288 fp32 143 (44), 2000 x 9001
// 84 (16). dx with two sweeps over the row, after ...
template <typename T, typename P>
__global__ void __launch_bounds__(1024) layer_norm_backward_long_kernel(LayerNormGradArgs a) {
  __shared__ GroupSums<2, 8> red;
  clear_sums(red);
  const float inv = 1.0f / static_cast<float>(a.cols);
  const P* w = static_cast<const P*>(a.weight);
  int parity = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, parity ^= 1) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
    const T* gr = static_cast<const T*>(a.dy) + row * a.lddy;
    T* dr = static_cast<T*>(a.dx) + row * a.lddx;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = to_f32(gr[c]) * (w != nullptr ? to_f32(w[c]) : 1.0f);
      s1 += g;
      s2 = fmaf(g, (to_f32(xr[c]) - mean) * rstd, s2);
    }
    float sums[2] = {s1, s2};
    group_sum(sums, red, parity);
    const float c1 = sums[0] * inv, c2 = sums[1] * inv;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = to_f32(gr[c]) * (w != nullptr ? to_f32(w[c]) : 1.0f);
      dr[c] = from_f32<T>(rstd * (g - c1 - (to_f32(xr[c]) - mean) * rstd * c2));
    }
  }
}

// ... the column sums, a thread per column over a range of rows.
template <typename T>
__global__ void __launch_bounds__(256) layer_norm_columns_kernel(LayerNormGradArgs a, long long rows_per_part) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.cols) return;
  const long long r0 = blockIdx.y * rows_per_part;
  const long long r1 = min(a.rows, r0 + rows_per_part);
  float dw = 0.0f, db = 0.0f;
#pragma unroll 4
  for (long long row = r0; row < r1; ++row) {
    const float dy = to_f32(static_cast<const T*>(a.dy)[row * a.lddy + c]);
    const float x = to_f32(static_cast<const T*>(a.x)[row * a.ldx + c]);
    dw = fmaf(dy, (x - a.mean[row]) * a.rstd[row], dw);
    db += dy;
  }
  float* out = a.partial + static_cast<size_t>(blockIdx.y) * 2 * a.cols;
  out[c] = dw;
  out[a.cols + c] = db;
}

// Add the blocks' partial rows column by column in a fixed order (0 rows: zeros).
constexpr int kJoinRows = 8;

template <typename P>
__global__ void __launch_bounds__(32 * kJoinRows) layer_norm_join_kernel(const float* __restrict__ partial, int parts,
                                                                         int cols, P* dweight, P* dbias) {
  __shared__ float sum[kJoinRows][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  if (c < 2 * cols) {
#pragma unroll 4
    for (int p = threadIdx.y; p < parts; p += kJoinRows) s += partial[static_cast<size_t>(p) * 2 * cols + c];
  }
  sum[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= 2 * cols) return;
#pragma unroll
  for (int r = 1; r < kJoinRows; ++r) s += sum[r][threadIdx.x];
  P* out = c < cols ? dweight : dbias;
  if (out != nullptr) out[c < cols ? c : c - cols] = from_f32<P>(s);
}

// The block for rows of `chunks` accesses with `ch` accesses per thread: false when more
// than max_threads threads would be needed.
bool pick_block(int chunks, int ch, int max_threads, dim3* block) {
  const int threads = (chunks + ch * 32 - 1) / (ch * 32) * 32;
  *block = threads == 32 ? dim3(32, kWarpRows) : dim3(threads, 1);
  return threads <= max_threads;
}

bool vec_ok(const void* p, long long ld, int cols, size_t elem, long long rows) {
  const int n = static_cast<int>(16 / elem);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && cols % n == 0 && (rows <= 1 || ld % n == 0);
}

// Blocks (or clusters) of a kernel that the current device holds at once. Asking costs
// more than the launch, so each thread keeps the last answer per kernel. Where a shape
// exceeds the 48 KB (static part included) that every kernel may use, the kernel's shared
// memory limit goes up first: always to the device's maximum, because the limit belongs to
// the kernel on the device and other threads launch other shapes under it.
struct Residency {
  int device = -1, threads = 0, cluster = 0;
  int raised = -1;  // the device on which this thread last raised the limit
  size_t smem = 0;
  int count = 0;
};

template <typename K>
cudaError_t raise_smem_limit(K kernel, int device) {
  int most = 0;
  cudaFuncAttributes attr;
  cudaError_t e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, device);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&attr, kernel);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              most - static_cast<int>(attr.sharedSizeBytes));
}

template <typename K>
cudaError_t residency(K kernel, Residency& last, dim3 block, size_t smem, int cluster, int num_sms, int* count) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const int threads = static_cast<int>(block.x * block.y);
  if (device != last.device || threads != last.threads || smem != last.smem || cluster != last.cluster) {
    if (smem > 40 * 1024 && last.raised != device) {
      if ((e = raise_smem_limit(kernel, device)) != cudaSuccess) return e;
      last.raised = device;
    }
    int n = 0;
    if (cluster > 1) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(cluster);
      cfg.blockDim = block;
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = cluster;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      // a cluster stays within a GPC: fewer blocks fit than of single ones
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    } else {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
      n *= num_sms;
    }
    if (e != cudaSuccess) return e;
    last.device = device;
    last.threads = threads;
    last.smem = smem;
    last.cluster = cluster;
    last.count = n > 0 ? n : 1;
  }
  *count = last.count;
  return cudaSuccess;
}

// (one call site per kernel, so that each has its own record)
#define QKVCTE_RESIDENT(kernel, block, smem, cluster, num_sms, count)          \
  ([&] {                                                                       \
    static thread_local Residency last;                                        \
    return residency(kernel, last, block, smem, cluster, num_sms, count);      \
  }())

template <typename Fm>
cudaError_t forward_launch(const LayerNormArgs& a, dim3 block, cudaStream_t s, int num_sms) {
  auto k = layer_norm_kernel<Fm>;
  const long long groups = (a.rows + block.y - 1) / block.y;
  const size_t smem = Fm::Forward::bytes(a.cols, block.x, block.y);
  int resident = 0;
  const cudaError_t e = QKVCTE_RESIDENT(k, block, smem, 1, num_sms, &resident);
  if (e != cudaSuccess) return e;
  // Eight times the resident blocks, but eight rows for each: with rows dealt out once, the
  // SMs that get less of the bandwidth finish last (32760 x 5120 bf16 118 us; 113, 106, 101
  // and 104 with 2, 4, 8 and 16 times).
  const long long grid = std::max<long long>(resident, std::min<long long>(8LL * resident, groups / 8));
  k<<<static_cast<int>(std::min(groups, grid)), block, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, typename P, int VEC, int CH, bool kKeep>
cudaError_t forward_go(const LayerNormArgs& a, dim3 block, cudaStream_t s, int num_sms) {
  if constexpr (VEC > 1) {
    if (a.cols == static_cast<int>(block.x) * CH * VEC)
      return forward_launch<Form<T, P, VEC, CH, kKeep, true>>(a, block, s, num_sms);
  }
  return forward_launch<Form<T, P, VEC, CH, kKeep, false>>(a, block, s, num_sms);
}

// Accesses per thread: one or two for rows of up to 32 (a warp) or 256 accesses, then four,
// eight (16 single elements) for long rows. More accesses per thread mean fewer warps per
// row, each of which pays for the reductions and addresses: 5120 bf16 columns on 160
// threads took 105 us for 32760 rows, on 320 threads 150 us. Rows off 16-byte boundaries
// (16000 x 5121 bf16) take 152 us where 5120 columns take 55: every element is a shared
// memory access and a store of its own.
template <typename T, typename P, int VEC>
cudaError_t forward_vec(const LayerNormArgs& a, cudaStream_t s, int num_sms) {
  dim3 block;
  const int chunks = a.cols / VEC;
  if (chunks <= 32 && pick_block(chunks, 1, 32, &block)) return forward_go<T, P, VEC, 1, true>(a, block, s, num_sms);
  if (chunks <= 256 && pick_block(chunks, 2, 256, &block)) return forward_go<T, P, VEC, 2, true>(a, block, s, num_sms);
  if (chunks <= 1024 || VEC > 1) {
    if (pick_block(chunks, 4, 512, &block)) return forward_go<T, P, VEC, 4, true>(a, block, s, num_sms);
  }
  if constexpr (VEC > 1) {
    if (pick_block(chunks, 8, 512, &block)) return forward_go<T, P, VEC, 8, false>(a, block, s, num_sms);
  } else {
    if (pick_block(chunks, 16, 512, &block)) return forward_go<T, P, VEC, 16, true>(a, block, s, num_sms);
  }
  auto k = layer_norm_long_kernel<T, P>;
  k<<<static_cast<int>(std::min<long long>(a.rows, 2 * num_sms)), 1024, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, typename P>
cudaError_t forward(const LayerNormArgs& a, cudaStream_t s, int num_sms) {
  constexpr int VEC = 16 / sizeof(T);
  const bool params = reinterpret_cast<uintptr_t>(a.weight) % 16 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  if (params && vec_ok(a.x, a.ldx, a.cols, sizeof(T), a.rows) && vec_ok(a.y, a.ldy, a.cols, sizeof(T), a.rows))
    return forward_vec<T, P, VEC>(a, s, num_sms);
  return forward_vec<T, P, 1>(a, s, num_sms);
}

template <typename P>
cudaError_t join(const LayerNormGradArgs& a, int parts, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((2 * a.cols + 31) / 32);
  cfg.blockDim = dim3(32, kJoinRows);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, layer_norm_join_kernel<P>, static_cast<const float*>(a.partial), parts, a.cols,
                            static_cast<P*>(a.dweight), static_cast<P*>(a.dbias));
}

template <typename Fm>
cudaError_t backward_launch(const LayerNormGradArgs& a, dim3 block, cudaStream_t s, int num_sms) {
  auto k = layer_norm_backward_kernel<Fm>;
  size_t smem = 2 * static_cast<size_t>(Fm::Backward::bytes(a.cols, block.x, block.y));
  const bool sums = a.partial != nullptr;
  if (sums) smem = std::max(smem, 2 * sizeof(float) * static_cast<size_t>(a.cols));
  const int cluster = sums ? kGradCluster : 1;
  int resident = 0;
  cudaError_t e = QKVCTE_RESIDENT(k, block, smem, cluster, num_sms, &resident);
  if (e != cudaSuccess) return e;
  if (sums) resident = std::min(resident, a.max_parts);
  const long long groups = (a.rows + block.y - 1) / block.y;
  const int grid = static_cast<int>(std::min<long long>((groups + cluster - 1) / cluster, resident)) * cluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k, a);
  return e != cudaSuccess || !sums ? e : join<typename Fm::P>(a, grid / cluster, s);
}

template <typename T, typename P, int VEC, int CH, bool kKeep>
cudaError_t backward_go(const LayerNormGradArgs& a, dim3 block, cudaStream_t s, int num_sms) {
  if constexpr (VEC > 1) {
    if (a.cols == static_cast<int>(block.x) * CH * VEC)
      return backward_launch<Form<T, P, VEC, CH, kKeep, true>>(a, block, s, num_sms);
  }
  return backward_launch<Form<T, P, VEC, CH, kKeep, false>>(a, block, s, num_sms);
}

template <typename T, typename P, int VEC>
cudaError_t backward_vec(const LayerNormGradArgs& a, cudaStream_t s, int num_sms) {
  dim3 block;
  const int chunks = a.cols / VEC;
  if (chunks <= 32 && pick_block(chunks, 1, 32, &block)) return backward_go<T, P, VEC, 1, true>(a, block, s, num_sms);
  if (chunks <= 256 && pick_block(chunks, 2, 256, &block)) return backward_go<T, P, VEC, 2, true>(a, block, s, num_sms);
  if constexpr (VEC > 1) {
    if (pick_block(chunks, 4, 256, &block)) return backward_go<T, P, VEC, 4, true>(a, block, s, num_sms);
    if (pick_block(chunks, 4, 512, &block)) return backward_go<T, P, VEC, 4, false>(a, block, s, num_sms);
  } else {
    if (chunks <= 1024 && pick_block(chunks, 4, 512, &block))
      return backward_go<T, P, VEC, 4, true>(a, block, s, num_sms);
    if (pick_block(chunks, 16, 512, &block)) return backward_go<T, P, VEC, 16, true>(a, block, s, num_sms);
  }
  // The column sums first: dx may overwrite dy or x.
  cudaError_t e = cudaSuccess;
  int parts = 0;
  if (a.partial != nullptr) {
    const int strips = (a.cols + 255) / 256;
    const long long want = std::max<long long>(1, static_cast<long long>(num_sms) * 8 / strips);
    const long long parts0 = std::min<long long>(std::min<long long>(want, a.max_parts), a.rows);
    const long long per = (a.rows + parts0 - 1) / parts0;
    parts = static_cast<int>((a.rows + per - 1) / per);
    layer_norm_columns_kernel<T><<<dim3(strips, parts), 256, 0, s>>>(a, per);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (a.dx != nullptr) {
    auto k = layer_norm_backward_long_kernel<T, P>;
    k<<<static_cast<int>(std::min<long long>(a.rows, 2 * num_sms)), 1024, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return a.partial == nullptr ? e : join<P>(a, parts, s);
}

template <typename T, typename P>
cudaError_t backward(const LayerNormGradArgs& a, bool sums, cudaStream_t s, int num_sms) {
  if (a.rows == 0) return sums ? join<P>(a, 0, s) : cudaSuccess;
  constexpr int VEC = 16 / sizeof(T);
  const bool params = reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
  if (params && vec_ok(a.x, a.ldx, a.cols, sizeof(T), a.rows) && vec_ok(a.dy, a.lddy, a.cols, sizeof(T), a.rows) &&
      (a.dx == nullptr || vec_ok(a.dx, a.lddx, a.cols, sizeof(T), a.rows)))
    return backward_vec<T, P, VEC>(a, s, num_sms);
  return backward_vec<T, P, 1>(a, s, num_sms);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, int dtype, int param_dtype, cudaStream_t s, int num_sms) {
  if (a.rows == 0) return cudaSuccess;
  const bool pf = param_dtype == QKV_CTE_DTYPE_FP32;
  switch (dtype) {
    case QKV_CTE_DTYPE_BF16:
      return pf ? forward<__nv_bfloat16, float>(a, s, num_sms) : forward<__nv_bfloat16, __nv_bfloat16>(a, s, num_sms);
    case QKV_CTE_DTYPE_FP16: return pf ? forward<__half, float>(a, s, num_sms) : forward<__half, __half>(a, s, num_sms);
    default: return forward<float, float>(a, s, num_sms);
  }
}

cudaError_t launch_layer_norm_backward(const LayerNormGradArgs& a, int dtype, int param_dtype, bool sums,
                                       cudaStream_t s, int num_sms) {
  const bool pf = param_dtype == QKV_CTE_DTYPE_FP32;
  switch (dtype) {
    case QKV_CTE_DTYPE_BF16:
      return pf ? backward<__nv_bfloat16, float>(a, sums, s, num_sms)
                : backward<__nv_bfloat16, __nv_bfloat16>(a, sums, s, num_sms);
    case QKV_CTE_DTYPE_FP16:
      return pf ? backward<__half, float>(a, sums, s, num_sms) : backward<__half, __half>(a, sums, s, num_sms);
    default: return backward<float, float>(a, sums, s, num_sms);
  }
}

}  // namespace qkvcte

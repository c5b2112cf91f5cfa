// Layer norm over the last dimension, forward and backward.
//
//   mu = mean(x), var = mean((x - mu)^2), r = 1 / sqrt(var + eps), xh = (x - mu) r
//   y  = xh * w + b
//   g  = dy * w,  dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Both passes are bound by memory (2 and 3 times the tensor). A row is held in the
// registers of one group of threads (a warp for short rows, a block for long ones), so
// it is read once; the variance is taken about the mean in a second sweep over the
// registers, never as a difference of large sums. The backward pass keeps its column
// sums dw and db in the registers of the same threads over all rows of the block, one
// partial row per block goes to the workspace, and a second kernel adds those in a
// fixed order (no atomics: the result does not depend on the schedule). Sums,
// statistics and gradients are fp32; x and the outputs are rounded once.
#include <algorithm>

#include "block_ops.h"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

namespace {

constexpr int kWarpRows = 4;  // rows (warps) per block of the warp-per-row form

// Sum over the group of threads that holds a row: a warp (blockDim.x == 32, no
// barrier) or the whole block. `slot` alternates between consecutive calls: a thread
// writes a slot again only after the barrier of the call in between, which every
// reader of the slot has reached.
__device__ __forceinline__ float group_sum(float v, float (*red)[32], int slot) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (blockDim.x == 32) return v;
  const int warps = blockDim.x >> 5;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[slot][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? red[slot][lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// VEC elements per access, CH accesses per thread: rows of up to CH * VEC * blockDim.x.
template <typename T, typename P, int VEC, int CH>
__global__ void __launch_bounds__(1024) layer_norm_kernel(LayerNormArgs a) {
  __shared__ float red[2][32];
  const float inv = 1.0f / static_cast<float>(a.cols);
  const P* w = static_cast<const P*>(a.weight);
  const P* b = static_cast<const P*>(a.bias);
  for (long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows;
       row += static_cast<long long>(gridDim.x) * blockDim.y) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
    T* yr = static_cast<T*>(a.y) + row * a.ldy;
    Vec<T, VEC> v[CH];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
      if (c < a.cols) v[i] = ld_once<T, VEC>(xr + c);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if ((i * blockDim.x + threadIdx.x) * VEC < a.cols) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) s += to_f32(v[i].v[j]);
      }
    }
    const float mean = group_sum(s, red, 0) * inv;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if ((i * blockDim.x + threadIdx.x) * VEC < a.cols) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = to_f32(v[i].v[j]) - mean;
          ss = fmaf(d, d, ss);
        }
      }
    }
    const float rstd = 1.0f / sqrtf(group_sum(ss, red, 1) * inv + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
      if (c < a.cols) {
        float wv[VEC], bv[VEC];
        if (w != nullptr) ld_params<P, VEC>(w + c, wv);
        if (b != nullptr) ld_params<P, VEC>(b + c, bv);
        Vec<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float xh = (to_f32(v[i].v[j]) - mean) * rstd;
          o.v[j] = from_f32<T>(fmaf(xh, w != nullptr ? wv[j] : 1.0f, b != nullptr ? bv[j] : 0.0f));
        }
        st_vec(yr + c, o);
      }
    }
  }
}

// Rows longer than the registers of a block: read three times (from L2 after the first).
template <typename T, typename P>
__global__ void __launch_bounds__(1024) layer_norm_long_kernel(LayerNormArgs a) {
  __shared__ float red[2][32];
  const float inv = 1.0f / static_cast<float>(a.cols);
  const P* w = static_cast<const P*>(a.weight);
  const P* b = static_cast<const P*>(a.bias);
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
    T* yr = static_cast<T*>(a.y) + row * a.ldy;
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) s += to_f32(xr[c]);
    const float mean = group_sum(s, red, 0) * inv;
    float ss = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float d = to_f32(xr[c]) - mean;
      ss = fmaf(d, d, ss);
    }
    const float rstd = 1.0f / sqrtf(group_sum(ss, red, 1) * inv + a.eps);
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

// Rows held in registers, columns fixed to threads; the block's column sums leave as one
// row of the workspace.
template <typename T, typename P, int VEC, int CH>
__global__ void __launch_bounds__(512) layer_norm_backward_kernel(LayerNormGradArgs a) {
  __shared__ float red[2][2][32];
  extern __shared__ float cols_sum[];  // [2][cols], only with several rows per block
  const float inv = 1.0f / static_cast<float>(a.cols);
  const P* w = static_cast<const P*>(a.weight);
  float dw[CH][VEC], db[CH][VEC];
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.0f;
  int parity = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y; row < a.rows;
       row += static_cast<long long>(gridDim.x) * blockDim.y, parity ^= 1) {
    const T* xr = static_cast<const T*>(a.x) + row * a.ldx;
    const T* gr = static_cast<const T*>(a.dy) + row * a.lddy;
    Vec<T, VEC> xv[CH], gv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
      if (c < a.cols) {
        xv[i] = ld_once<T, VEC>(xr + c);
        gv[i] = ld_once<T, VEC>(gr + c);
      }
    }
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
      if (c < a.cols) {
        float wv[VEC];
        if (w != nullptr) ld_params<P, VEC>(w + c, wv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float dy = to_f32(gv[i].v[j]);
          const float xh = (to_f32(xv[i].v[j]) - mean) * rstd;
          const float g = w != nullptr ? dy * wv[j] : dy;
          s1 += g;
          s2 = fmaf(g, xh, s2);
          dw[i][j] = fmaf(dy, xh, dw[i][j]);
          db[i][j] += dy;
        }
      }
    }
    if (a.dx == nullptr) continue;  // uniform over the grid
    const float c1 = group_sum(s1, red[0], parity) * inv;
    const float c2 = group_sum(s2, red[1], parity) * inv;
    T* dr = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = (i * blockDim.x + threadIdx.x) * VEC;
      if (c < a.cols) {
        float wv[VEC];
        if (w != nullptr) ld_params<P, VEC>(w + c, wv);
        Vec<T, VEC> o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float dy = to_f32(gv[i].v[j]);
          const float xh = (to_f32(xv[i].v[j]) - mean) * rstd;
          const float g = w != nullptr ? dy * wv[j] : dy;
          o.v[j] = from_f32<T>(rstd * (g - c1 - xh * c2));
        }
        st_vec(dr + c, o);
      }
    }
  }
  if (a.partial == nullptr) return;
  float* out = a.partial + static_cast<size_t>(blockIdx.x) * 2 * a.cols;
  if (blockDim.y > 1) {  // the block's rows (warps) one after the other, in order
    for (int r = 0; r < static_cast<int>(blockDim.y); ++r) {
      if (static_cast<int>(threadIdx.y) == r) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int c = (i * blockDim.x + threadIdx.x) * VEC;
          if (c < a.cols) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              cols_sum[c + j] = r == 0 ? dw[i][j] : cols_sum[c + j] + dw[i][j];
              cols_sum[a.cols + c + j] = r == 0 ? db[i][j] : cols_sum[a.cols + c + j] + db[i][j];
            }
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < 2 * a.cols; c += blockDim.x * blockDim.y)
      out[c] = cols_sum[c];
    return;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * VEC;
    if (c < a.cols) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        out[c + j] = dw[i][j];
        out[a.cols + c + j] = db[i][j];
      }
    }
  }
}

// Rows longer than the registers: dx with two sweeps over the row ...
template <typename T, typename P>
__global__ void __launch_bounds__(1024) layer_norm_backward_long_kernel(LayerNormGradArgs a) {
  __shared__ float red[2][2][32];
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
    const float c1 = group_sum(s1, red[0], parity) * inv;
    const float c2 = group_sum(s2, red[1], parity) * inv;
    for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
      const float g = to_f32(gr[c]) * (w != nullptr ? to_f32(w[c]) : 1.0f);
      dr[c] = from_f32<T>(rstd * (g - c1 - (to_f32(xr[c]) - mean) * rstd * c2));
    }
  }
}

// ... and the column sums, a thread per column over a range of rows.
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

// Threads and accesses per thread for a row of `chunks` accesses: a warp when a warp
// holds it, else the fewest accesses per thread (a power of two from `ch0`) with which
// `max_threads` threads hold it. 0: it does not fit.
int pick_accesses(int chunks, int ch0, int ch_max, int max_threads, dim3* block) {
  if (chunks <= 32 * ch0) {
    int ch = 1;
    while (32 * ch < chunks) ch *= 2;
    *block = dim3(32, kWarpRows);
    return ch;
  }
  for (int ch = ch0; ch <= ch_max; ch *= 2) {
    const int threads = (chunks + ch * 32 - 1) / (ch * 32) * 32;
    if (threads <= max_threads) {
      *block = dim3(threads, 1);
      return ch;
    }
  }
  return 0;
}

bool vec_ok(const void* p, long long ld, int cols, size_t elem, long long rows) {
  const int n = static_cast<int>(16 / elem);
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && cols % n == 0 && (rows <= 1 || ld % n == 0);
}

template <typename K>
int resident_grid(K kernel, dim3 block, size_t smem, int num_sms, long long work) {
  int per_sm = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, static_cast<int>(block.x * block.y), smem) !=
          cudaSuccess ||
      per_sm < 1)
    per_sm = 1;
  return static_cast<int>(std::min<long long>(static_cast<long long>(per_sm) * num_sms, work));
}

template <typename T, typename P, int VEC, int CH>
cudaError_t forward_go(const LayerNormArgs& a, dim3 block, cudaStream_t s, int num_sms) {
  auto k = layer_norm_kernel<T, P, VEC, CH>;
  const long long groups = (a.rows + block.y - 1) / block.y;
  k<<<resident_grid(k, block, 0, num_sms, groups), block, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, typename P, int VEC>
cudaError_t forward_vec(const LayerNormArgs& a, cudaStream_t s, int num_sms) {
  dim3 block;
  switch (pick_accesses(a.cols / VEC, 4, VEC == 1 ? 16 : 8, 1024, &block)) {
    case 1: return forward_go<T, P, VEC, 1>(a, block, s, num_sms);
    case 2: return forward_go<T, P, VEC, 2>(a, block, s, num_sms);
    case 4: return forward_go<T, P, VEC, 4>(a, block, s, num_sms);
    case 8: return forward_go<T, P, VEC, 8>(a, block, s, num_sms);
    case 16:
      if constexpr (VEC == 1) return forward_go<T, P, VEC, 16>(a, block, s, num_sms);
    default: break;
  }
  auto k = layer_norm_long_kernel<T, P>;
  k<<<resident_grid(k, dim3(1024), 0, num_sms, a.rows), 1024, 0, s>>>(a);
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

template <typename T, typename P, int VEC, int CH>
cudaError_t backward_go(const LayerNormGradArgs& a, dim3 block, cudaStream_t s, int num_sms) {
  auto k = layer_norm_backward_kernel<T, P, VEC, CH>;
  const size_t smem = block.y > 1 && a.partial != nullptr ? 2 * sizeof(float) * static_cast<size_t>(a.cols) : 0;
  long long groups = (a.rows + block.y - 1) / block.y;
  if (a.partial != nullptr) groups = std::min<long long>(groups, a.max_parts);
  const int grid = resident_grid(k, block, smem, num_sms, groups);
  k<<<grid, block, smem, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess || a.partial == nullptr ? e : join<P>(a, grid, s);
}

template <typename T, typename P, int VEC>
cudaError_t backward_vec(const LayerNormGradArgs& a, cudaStream_t s, int num_sms) {
  dim3 block;
  // two 16-byte accesses per thread and tensor keep dw and db (32 fp32) in registers
  // without spilling; four where the row needs them
  switch (pick_accesses(a.cols / VEC, VEC == 1 ? 4 : 2, VEC == 1 ? 16 : 4, 512, &block)) {
    case 1: return backward_go<T, P, VEC, 1>(a, block, s, num_sms);
    case 2: return backward_go<T, P, VEC, 2>(a, block, s, num_sms);
    case 4: return backward_go<T, P, VEC, 4>(a, block, s, num_sms);
    case 8:
      if constexpr (VEC == 1) return backward_go<T, P, VEC, 8>(a, block, s, num_sms);
    case 16:
      if constexpr (VEC == 1) return backward_go<T, P, VEC, 16>(a, block, s, num_sms);
    default: break;
  }
  cudaError_t e = cudaSuccess;
  if (a.dx != nullptr) {
    auto k = layer_norm_backward_long_kernel<T, P>;
    k<<<resident_grid(k, dim3(1024), 0, num_sms, a.rows), 1024, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (a.partial == nullptr) return e;
  const int strips = (a.cols + 255) / 256;
  const long long want = std::max<long long>(1, static_cast<long long>(num_sms) * 8 / strips);
  const long long parts0 = std::min<long long>(std::min<long long>(want, a.max_parts), a.rows);
  const long long per = (a.rows + parts0 - 1) / parts0;
  const int parts = static_cast<int>((a.rows + per - 1) / per);
  layer_norm_columns_kernel<T><<<dim3(strips, parts), 256, 0, s>>>(a, per);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return join<P>(a, parts, s);
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

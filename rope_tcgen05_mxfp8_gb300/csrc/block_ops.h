// Internal interfaces of the block operators (layer norm, rotary positions with several
// axes, the product with its epilogue): arguments and launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace qkvcte {

// Layer norm. Strides are in elements; the types of x/y and of the parameters are
// QKV_CTE_DTYPE_* values.
struct LayerNormArgs {
  const void* x;
  long long ldx;
  const void* weight;  // [cols] or null: 1
  const void* bias;    // [cols] or null: 0
  void* y;
  long long ldy;
  float* mean;  // [rows] or null
  float* rstd;  // [rows] or null
  long long rows;
  int cols;
  float eps;
};

struct LayerNormGradArgs {
  const void* dy;
  long long lddy;
  const void* x;
  long long ldx;
  const void* weight;  // [cols] or null: 1
  const float* mean;
  const float* rstd;
  void* dx;  // or null
  long long lddx;
  void* dweight;  // [cols] or null
  void* dbias;    // [cols] or null
  float* partial;  // [parts][2][cols] partial column sums, or null: no dweight or dbias
  int max_parts;
  long long rows;
  int cols;
};

// Partial rows of column sums the backward pass keeps apart (bounds its workspace).
constexpr int kLayerNormMaxParts = 128;

cudaError_t launch_layer_norm(const LayerNormArgs& a, int dtype, int param_dtype, cudaStream_t s, int num_sms);
// `sums`: dweight and/or dbias are wanted (with no rows they are zeros).
cudaError_t launch_layer_norm_backward(const LayerNormGradArgs& a, int dtype, int param_dtype, bool sums,
                                       cudaStream_t s, int num_sms);

// Rotary positions with several axes.
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeMaxPairs = 256;

// What a plan fixes: the head's pairs, their axes and steps.
struct RopePairs {
  int d, n_axes;
  int first_pair[kRopeMaxAxes];               // first pair of each axis
  unsigned long long step[kRopeMaxPairs];     // turns per position, as a binary fraction of a turn
};

struct RopeArgs : RopePairs {
  int batch, seq, heads;
  const int* positions;         // [seq, n_axes] per batch, or null
  long long pos_batch_stride;   // 0: one set for every batch
  const int* grids;             // [batch, n_axes], or null
  const void* x;
  void* y;
  long long xb, xs, xh, yb, ys, yh;  // strides of batch, row and head in elements
  int inverse;
};

cudaError_t launch_rope_apply(const RopeArgs& a, int dtype, bool rotate_half, cudaStream_t s);
// cos_t, sin_t: fp32 [batch * seq, d], 8-byte aligned for interleaved pairs.
cudaError_t launch_rope_tables(const RopeArgs& a, float* cos_t, float* sin_t, bool rotate_half, cudaStream_t s);

// The product's epilogue beyond scale and bias (see linear_epilogue.cuh).
struct LinearEpilogue {
  int act;                // QKV_CTE_ACT_*
  int dtype;              // of the residual and the output
  const uint16_t* gate;   // [N] bf16, or null
  const void* residual;   // or null
  long long ldr;
  void* out;
  long long ldo;
  int wide;               // residual and output rows start on 32-byte boundaries
  int pairs;              // ... on boundaries of two elements
};

// The product's channel-major form (linear_few.cu).
struct LinearFewArgs {
  const float* a_scale;
  const float* w_col_scale;  // or null
  const uint16_t* bias;      // or null
  const uint8_t* w_sf;       // [N, k_blocks]
  int T, N;
  int k_blocks;              // K / 32
  int k_stages;              // ceil(K / 128)
  int split;                 // CTAs of a cluster that share a tile's K blocks: 1, 2, 4 or 8, <= k_stages
  uint32_t flags;
  uint32_t* status;
  LinearEpilogue lin;
};

}  // namespace qkvcte

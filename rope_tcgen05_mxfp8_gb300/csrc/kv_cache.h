// Internal interfaces of the 8-bit key/value cache: writing, reading back, attention.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace qkvcte {

// The pool and the pages of each sequence. Page p holds, for each head, block_tokens rows of
// d e4m3 codes and one UE8M0 scale for K and for V.
struct CachePool {
  uint8_t* k;
  uint8_t* k_sf;
  uint8_t* v;
  uint8_t* v_sf;
  const int* table;        // [batch, max_blocks] pages, or null: sequence b owns pages b * max_blocks + ...
  long long table_stride;
  long long pages;
  int max_blocks;
  int heads, d;
  int log_bt;              // block_tokens = 1 << log_bt
};

// A [batch, seq, heads, d] tensor: strides in elements, lanes contiguous.
struct HeadsTensor {
  void* p;
  long long sb, ss, sh;
};

struct CacheCopyArgs {
  CachePool pool;
  HeadsTensor k, v;      // a null p: not wanted
  const int* starts;     // [batch]
  const int* counts;     // write: [batch] or null (seq)
  const int* lengths;    // read: [batch]
  int batch, seq;
  int blocks;            // pages a sequence's rows can touch: ceil(seq / block_tokens) + 1
  int wide;              // every row starts on a 16-byte boundary
};

cudaError_t launch_cache_write(const CacheCopyArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache_read(const CacheCopyArgs& a, int dtype, cudaStream_t s);

struct CacheAttentionArgs {
  CachePool pool;
  HeadsTensor q, out;
  float* lse;            // [batch, seq, q_heads] or null
  const int* lengths;    // [batch]
  const int* counts;     // [batch] or null (seq)
  int batch, seq, q_heads, group;  // group: query heads per key head
  int row_tiles;         // tiles of the seq * group rows of a (batch, key head): of 16, or of 512
  int splits;            // parts of the keys
  float scale_log2;      // softmax scale * log2(e)
  int causal, window;    // window 0: none
  int wide;              // rows of q start on 16-byte boundaries
  int wide32, wide32_out;  // rows of q, of out start on 32-byte boundaries
  float* part_o;         // splits > 1: [splits][batch * seq * q_heads][d], each part normalised
  float* part_lse;       // splits > 1: [splits][batch * seq * q_heads], base 2
  uint32_t* status;
  uint32_t flags;
};

// Rows a block takes of the form for few queries, a pair of blocks of the form on tcgen05.
constexpr int kCacheFewRows = 16;
constexpr int kCacheTileRows = 512;

cudaError_t launch_cache_attention_few(const CacheAttentionArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_cache_attention_tiles(const CacheAttentionArgs& a, int dtype, cudaStream_t s);
// Joins the parts of the keys.
cudaError_t launch_cache_attention_join(const CacheAttentionArgs& a, int dtype, cudaStream_t s);

}  // namespace qkvcte

// Writing keys and values to the 8-bit cache, and reading them back.
//
// A scale belongs to one page and head: 2^(E - 127), E the smallest exponent that brings the
// largest magnitude to at most 448. Scales are powers of two because floating codes gain
// nothing from a finer one (their relative step is the same everywhere between 2^-6 and
// 448), and because everything about them is then exact: x * 2^(127 - E) rounds once, in the
// conversion to e4m3, and codes that were in the page before move to a larger scale by an
// exponent (rounding again only where they fall under 2^-6).
//
// A group of threads owns one (page, head) of K or of V: it holds the page's new tokens in
// registers (64 elements a thread), finds their largest magnitude as a maximum of bit
// patterns (infinities and NaN order above the rest: they make the scale 255, a NaN for the
// whole page and head), joins it with the old scale where the page holds earlier tokens, and
// writes codes. Each element is read once and each code written once: both kernels are bound by
// memory. 32760 tokens, 40 heads of 128, bf16: written in 167 us (6.0 TB/s, 0.89 of the copy
// rate; floor 148), read in 150 (6.7 TB/s). One token for each of 4 sequences: 19 us a call, the
// host's part.
#include "kv_cache.cuh"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

namespace {

constexpr int kVecs = 8;        // vectors of 8 elements per thread
constexpr int kWarpItems = 8;   // items of one warp each per block

// Eight elements as they lie in memory.
template <typename T>
struct Eight {
  static constexpr int WORDS = 2 * sizeof(T);
  uint32_t w[WORDS];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const T* p, bool wide) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < WORDS / 4; ++i) {
        const Vec<uint32_t, 4> r = ld_once<uint32_t, 4>(reinterpret_cast<const uint32_t*>(p) + 4 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = r.w[j];
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(p[i]);
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = h[2 * i] | static_cast<uint32_t>(h[2 * i + 1]) << 16;
    }
  }
  __device__ __forceinline__ void store(T* p, bool wide) const {
    if (wide) {
#pragma unroll
      for (int i = 0; i < WORDS / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = __uint_as_float(w[i]);
    } else {
      uint16_t* h = reinterpret_cast<uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h[2 * i] = static_cast<uint16_t>(w[i]);
        h[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
      }
    }
  }
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
  // Largest pattern without signs: of both halves of a word for 2-byte types.
  __device__ __forceinline__ uint32_t max_bits(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      if constexpr (sizeof(T) == 4)
        m = max(m, w[i] & 0x7FFFFFFFu);
      else
        m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    }
    return m;
  }
};

// The bits of the largest magnitude as fp32.
template <typename T>
__device__ __forceinline__ uint32_t as_f32_bits(uint32_t m) {
  if constexpr (sizeof(T) == 4) return m;
  const uint32_t top = max(m & 0xFFFFu, m >> 16);
  return __float_as_uint(unpack_pair<T>(top).x) & 0x7FFFFFFFu;
}

// One item: a page and head of K (blockIdx.y 0) or V. Blocks walk the heads first: a token's
// heads lie side by side.
struct CopyItem {
  int b, h;
  long long blk, page;
  long long base;   // token of the page's first slot
  long long start;

  __device__ __forceinline__ CopyItem(const CacheCopyArgs& a, long long item) {
    h = static_cast<int>(item % a.pool.heads);
    item /= a.pool.heads;
    b = static_cast<int>(item / a.blocks);
    start = __ldg(a.starts + b);
    blk = (start >> a.pool.log_bt) + item % a.blocks;
    base = blk << a.pool.log_bt;
    page = cache_page(a.pool, b, blk);
  }
};

// kWarp: a warp per item, several items per block (pages of up to 2048 elements per head); else
// a block per item.
template <typename T, bool kWarp>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheCopyArgs a, long long items) {
  __shared__ uint32_t warp_max[8];
  const int group = kWarp ? 32 : static_cast<int>(blockDim.x);
  const int tid = kWarp ? static_cast<int>(threadIdx.x) & 31 : static_cast<int>(threadIdx.x);
  const long long item = kWarp ? static_cast<long long>(blockIdx.x) * kWarpItems + (threadIdx.x >> 5)
                               : static_cast<long long>(blockIdx.x);
  if (item >= items) return;
  const HeadsTensor& src = blockIdx.y == 0 ? a.k : a.v;
  if (src.p == nullptr) return;
  const CopyItem it(a, item);
  int count = a.counts != nullptr ? __ldg(a.counts + it.b) : a.seq;
  count = count < 0 ? 0 : count > a.seq ? a.seq : count;
  const long long end = it.start + count;
  const int bt = 1 << a.pool.log_bt;
  // slots [lo, hi) of the page receive tokens
  const int lo = it.start > it.base ? static_cast<int>(it.start - it.base) : 0;
  const int hi = end - it.base < bt ? static_cast<int>(end - it.base < 0 ? 0 : end - it.base) : bt;
  if (it.page < 0 || hi <= lo) return;  // the same for the whole group

  const int d8 = a.pool.d >> 3;                       // vectors per token
  const int magic = (65536 + d8 - 1) / d8;            // u / d8 for u < 4096, d8 <= 16
  const int vecs = bt * d8;
  const T* x = static_cast<const T*>(src.p) + it.b * src.sb + it.h * src.sh;
  Eight<T> e[kVecs];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int u = tid + i * group;
    const int slot = (u * magic) >> 16;
    e[i].zero();
    if (u < vecs && slot >= lo && slot < hi)
      e[i].load(x + (it.base + slot - it.start) * src.ss + 8 * (u - slot * d8), a.wide);
  }
#pragma unroll
  for (int i = 0; i < kVecs; ++i) top = e[i].max_bits(top);
  top = as_f32_bits<T>(top);
  top = __reduce_max_sync(0xffffffffu, top);
  const size_t ph = static_cast<size_t>(it.page) * a.pool.heads + it.h;
  uint8_t* sf = (blockIdx.y == 0 ? a.pool.k_sf : a.pool.v_sf) + ph;
  const int old = lo > 0 ? *sf : 0;  // the page's earlier tokens
  if constexpr (!kWarp) {
    if ((tid & 31) == 0) warp_max[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < group >> 5; ++w) top = max(top, warp_max[w]);
  } else {
    __syncwarp();
  }
  const int fresh = scale_exponent(top);
  const int now = fresh > old ? fresh : old;
  if (tid == 0 && now != old) *sf = static_cast<uint8_t>(now);

  uint8_t* codes = (blockIdx.y == 0 ? a.pool.k : a.pool.v) + (ph << a.pool.log_bt) * a.pool.d;
  const bool nan = now == kScaleNan;
  const float f = nan ? 0.0f : scale_value(254 - now);  // 2^(127 - now)
  const int shift = now - old;
  const bool move = lo > 0 && !nan && shift > 0;
  // shifts past 20 leave nothing of any code
  const float back = scale_value(127 - (shift > 20 ? 20 : shift));
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int u = tid + i * group;
    const int slot = (u * magic) >> 16;
    if (u >= vecs || slot >= hi) continue;
    uint2* to = reinterpret_cast<uint2*>(codes + 8 * static_cast<size_t>(u));
    uint2 c;
    if (slot >= lo) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = e[i].pair(j);
        w[j] = f32_to_codes(v.x * f, v.y * f);
      }
      c = nan ? make_uint2(0, 0) : make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
      *to = c;
    } else if (move) {
      c = *to;
      uint32_t w[4] = {c.x, c.x >> 16, c.y, c.y >> 16};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = half2_to_f32(codes_to_half2(w[j]));
        w[j] = f32_to_codes(v.x * back, v.y * back);
      }
      *to = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
  }
}

template <typename T, bool kWarp>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheCopyArgs a, long long items) {
  const int group = kWarp ? 32 : static_cast<int>(blockDim.x);
  const int tid = kWarp ? static_cast<int>(threadIdx.x) & 31 : static_cast<int>(threadIdx.x);
  const long long item = kWarp ? static_cast<long long>(blockIdx.x) * kWarpItems + (threadIdx.x >> 5)
                               : static_cast<long long>(blockIdx.x);
  if (item >= items) return;
  const HeadsTensor& dst = blockIdx.y == 0 ? a.k : a.v;
  if (dst.p == nullptr) return;
  const CopyItem it(a, item);
  const int bt = 1 << a.pool.log_bt;
  const long long end = it.start + a.seq;
  const int lo = it.start > it.base ? static_cast<int>(it.start - it.base) : 0;
  const int hi = end - it.base < bt ? static_cast<int>(end - it.base < 0 ? 0 : end - it.base) : bt;
  if (hi <= lo) return;
  const long long length = __ldg(a.lengths + it.b);
  // slots below `live` hold tokens; the rest of the rows are zeros
  const int live = it.page < 0 || length <= it.base ? 0 : length - it.base < bt ? static_cast<int>(length - it.base) : bt;

  const int d8 = a.pool.d >> 3;
  const int magic = (65536 + d8 - 1) / d8;
  const int vecs = bt * d8;
  const size_t ph = static_cast<size_t>(it.page < 0 ? 0 : it.page) * a.pool.heads + it.h;
  const uint8_t* codes = (blockIdx.y == 0 ? a.pool.k : a.pool.v) + (ph << a.pool.log_bt) * a.pool.d;
  uint2 c[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int u = tid + i * group;
    const int slot = (u * magic) >> 16;
    c[i] = make_uint2(0, 0);
    if (u < vecs && slot >= lo && slot < hi && slot < live) c[i] = *reinterpret_cast<const uint2*>(codes + 8 * static_cast<size_t>(u));
  }
  const float f = live > 0 ? scale_value((blockIdx.y == 0 ? a.pool.k_sf : a.pool.v_sf)[ph]) : 0.0f;
  T* y = static_cast<T*>(dst.p) + it.b * dst.sb + it.h * dst.sh;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int u = tid + i * group;
    const int slot = (u * magic) >> 16;
    if (u >= vecs || slot < lo || slot >= hi) continue;
    const uint32_t w[4] = {c[i].x, c[i].x >> 16, c[i].y, c[i].y >> 16};
    Eight<T> e;
    const float g = slot < live ? f : 0.0f;  // (a scale that is NaN leaves rows past the end alone)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = half2_to_f32(codes_to_half2(w[j]));
      e.set_pair(j, make_float2(v.x * g, v.y * g));
    }
    e.store(y + (it.base + slot - it.start) * dst.ss + 8 * (u - slot * d8), a.wide);
  }
}

template <typename T, bool kRead>
cudaError_t launch_copy(const CacheCopyArgs& a, cudaStream_t s) {
  const long long items = static_cast<long long>(a.batch) * a.blocks * a.pool.heads;
  const int threads = ((a.pool.d << a.pool.log_bt) / (8 * kVecs) + 31) / 32 * 32;
  if (threads == 32) {
    const dim3 grid(static_cast<unsigned>((items + kWarpItems - 1) / kWarpItems), 2);
    if (kRead)
      cache_read_kernel<T, true><<<grid, 32 * kWarpItems, 0, s>>>(a, items);
    else
      cache_write_kernel<T, true><<<grid, 32 * kWarpItems, 0, s>>>(a, items);
  } else {
    const dim3 grid(static_cast<unsigned>(items), 2);
    if (kRead)
      cache_read_kernel<T, false><<<grid, threads, 0, s>>>(a, items);
    else
      cache_write_kernel<T, false><<<grid, threads, 0, s>>>(a, items);
  }
  return cudaGetLastError();
}

template <bool kRead>
cudaError_t launch_copy_type(const CacheCopyArgs& a, int dtype, cudaStream_t s) {
  switch (dtype) {
    case QKV_CTE_DTYPE_BF16: return launch_copy<__nv_bfloat16, kRead>(a, s);
    case QKV_CTE_DTYPE_FP16: return launch_copy<__half, kRead>(a, s);
    case QKV_CTE_DTYPE_FP32: return launch_copy<float, kRead>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_cache_write(const CacheCopyArgs& a, int dtype, cudaStream_t s) { return launch_copy_type<false>(a, dtype, s); }
cudaError_t launch_cache_read(const CacheCopyArgs& a, int dtype, cudaStream_t s) { return launch_copy_type<true>(a, dtype, s); }

}  // namespace qkvcte

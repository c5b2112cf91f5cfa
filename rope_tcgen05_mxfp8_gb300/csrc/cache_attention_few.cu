// Attention of few queries over the 8-bit cache, and the joining of the keys' parts.
//
//   z_t = c q . k_t,  o = sum_t 2^z_t v_t / sum_t 2^z_t
// with c = scale log2(e) and running references per row: one pass over the keys.
//
// With a few query rows per key head (a token of each sequence, times the query heads that
// share a key head) the cache is read once and the read is what counts. A warp takes 32 keys
// at a time and multiplies them with up to 16 rows by warp-level tensor instructions
// (m16n8k16, fp16 in, fp32 out): the codes become fp16 exactly, and the instruction wants
// them in registers, where the global loads put them. No shared memory, no barrier and no
// conversion pass stands between memory and the product. tcgen05 would want the same codes
// converted and stored to shared memory first, for a tile whose 128 rows would be mostly
// padding (17 rows over 4096 keys, 40 heads: 26 us here, 53 there).
//
// What bounds it: 4 sequences of 32760 tokens, 40 heads of 128, one row each (1.34 GB) take 273 us,
// 4.9 TB/s of 6.8: the warps' chains of product, maximum, exponential and product, some 900
// instructions per 8 KB. More warps did not help (8 rows a tile in 168 or 128 registers: 276 and
// 295 us against 278 at the time), nor did integer operations in place of the conversion
// instructions (321). One token over 512 keys takes 9.4 us, latencies alone. Keys are divided among
// blocks by waves (see the host's attention_shape) and the parts joined by a second, small kernel.
//
// Layouts. Lane 4g + t holds column g of the B operand and rows g, g + 8 of A and C.
//   Scores: B's column g is key g; a lane reads 16-byte pieces t, t + 4 of its key's row, so
//   an instruction's 16 contracted lanes are bytes 4w .. 4w + 3 of the four lanes' pieces
//   (the order of a contraction is free; the queries are loaded in the same one).
//   Values: B's rows are keys 2t, 2t + 1, 2t + 8, 2t + 9, as the scores come out; a lane reads
//   the 16-byte piece g of those four keys, byte j of it being column g of the j-th of 16
//   products: its output columns are 16 g + j.
//
// Numerics. Queries are fp16 after a power of two per row (exact but for what is 2^-28 of the
// row's largest), codes are exact, products and sums fp32. Each key's block scales multiply
// its score and its weight in fp32; weights are rounded to fp16 (by 2^-11 at most; the product takes
// no more digits) with their value scale 2^x_t. While the value scales met lie within 2^12 of
// one another, a weight is 2^(z_t - m + x_t - x), m the row's maximum of z_t and x the largest
// x_t. Beyond, that would take the digits of weights that matter, for the sake of large values that
// the row does not see or whose weight is negligible: a weight is then 2^(z_t + x_t - m), m the row's
// own maximum of that over the keys it sees, and the sum of the 2^z_t has a reference and exponentials
// of its own (297 us for the 273 above, were it done all the time); both references are whole numbers
// then, so that their difference is exact however large they are. Held 2^14 above, the row's largest
// weight is 2^2 or more: down to 2^-16 of it weights keep fp16's digits, and what is 2^-27 of it is
// lost. While scales lie near, a key that is all a row sees has a weight of just 2^(14 + x_t - x), and
// its value comes out as it is.
#include <type_traits>

#include "kv_cache.cuh"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

namespace {

constexpr int kFewWarps = 4;
constexpr int kFewKeys = 32;       // keys a warp takes at a time
constexpr int kWeightBias = 14;    // weights are held 2^14 above their value
constexpr int kFewNear = 12;       // binary orders of value scales that share a reference
constexpr int kPitch = 132;        // floats per row of the warps' partial outputs (banks)

__device__ __forceinline__ void mma_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // 2 ulp; below 2^-126 zero (one instruction, not four)
  return y;
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Where 16 keys lie: their page (or none) and both scales.
struct KeyGroup {
  long long row;   // (page * heads + head) * block_tokens + slot, or -1
  int ek, ev;

  // `entry`: the table's, loaded an iteration earlier
  __device__ __forceinline__ void find(const CachePool& p, int entry, int h, int key) {
    row = -1;
    ek = ev = 1;
    if (entry >= 0 && entry < p.pages) {
      const long long ph = static_cast<long long>(entry) * p.heads + h;
      row = (ph << p.log_bt) + (key & ((1 << p.log_bt) - 1));
      ek = __ldg(p.k_sf + ph);
      ev = __ldg(p.v_sf + ph);
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kFewWarps * 32, 2) cache_attention_few_kernel(const CacheAttentionArgs a) {
  __shared__ float s_o[kFewWarps][kCacheFewRows][kPitch];
  __shared__ float s_m[kFewWarps][kCacheFewRows], s_x[kFewWarps][kCacheFewRows], s_l[kFewWarps][kCacheFewRows];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  long long item = blockIdx.x;
  const int split = static_cast<int>(item % a.splits);
  item /= a.splits;
  const int h = static_cast<int>(item % a.pool.heads);
  item /= a.pool.heads;
  const int tile = static_cast<int>(item % a.row_tiles);
  const int b = static_cast<int>(item / a.row_tiles);
  const int rows = a.seq * a.group;  // of this key head
  const int r0 = tile * kCacheFewRows;
  const int pieces = a.pool.d >> 4;  // 16-byte pieces of a code row

  // what the tile's rows see: from the first row's first key to the last row's last
  const Visible vis(a, b);
  const int s_first = r0 / a.group;
  int s_last = (r0 + kCacheFewRows - 1) / a.group;
  if (s_last > vis.count - 1) s_last = vis.count - 1;
  const int lo = vis.lo(a, s_first);
  const int hi = s_first > s_last ? 0 : vis.hi(a, s_last);
  const int c_begin = lo / kFewKeys, c_end = hi > lo ? (hi + kFewKeys - 1) / kFewKeys : c_begin;
  const int n_chunks = c_end - c_begin;
  const int c0 = c_begin + static_cast<int>(static_cast<long long>(n_chunks) * split / a.splits);
  const int c1 = c_begin + static_cast<int>(static_cast<long long>(n_chunks) * (split + 1) / a.splits);

  // queries: rows g and g + 8, elements 64 i + 16 t + 4 w .. + 3
  uint32_t qf[8][4];
  float coef[2];
  int row_lo[2], row_hi[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = r0 + g + 8 * k;
    const int s = r / a.group;
    const bool live = r < rows && s < vis.count;
    row_lo[k] = live ? vis.lo(a, s) : 0;
    row_hi[k] = live ? vis.hi(a, s) : 0;
    const T* p = static_cast<const T*>(a.q.p) + b * a.q.sb + s * a.q.ss + (h * a.group + r % a.group) * a.q.sh;
    float x[32];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const T* e = p + 64 * i + 16 * t;
      const bool there = live && 4 * i + t < pieces;
      if (a.wide) {
        Vec<T, 8> v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[k].w[j] = 0;
        if (there) {
          v[0] = *reinterpret_cast<const Vec<T, 8>*>(e);
          v[1] = *reinterpret_cast<const Vec<T, 8>*>(e + 8);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 f = v[j >> 2].pair(j & 3);
          x[16 * i + 2 * j] = f.x;
          x[16 * i + 2 * j + 1] = f.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) x[16 * i + j] = there ? to_f32(e[j]) : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int f = query_factor_field(top);
    const float up = scale_value(f);
    coef[k] = query_coef(top, f, a.scale_log2);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      qf[n][k] = pack_pair<__half>(make_float2(x[4 * n] * up, x[4 * n + 1] * up));
      qf[n][2 + k] = pack_pair<__half>(make_float2(x[4 * n + 2] * up, x[4 * n + 3] * up));
    }
  }
  // keys of [all_lo, all_hi) are seen by every live row
  const int all_lo = vis.lo(a, s_last < 0 ? 0 : s_last), all_hi = vis.hi(a, s_first);

  float o[16][4];
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[j][k] = 0.0f;
  // references, minus infinity before a key is seen: m of the weights (while scales lie near without
  // the largest of them, and the sum's too), mz of the sum where they lie apart; the sum
  float m[2] = {-INFINITY, -INFINITY}, mz[2], l[2] = {0.0f, 0.0f};
  int most = 1, least = kScaleNan;  // exponents of the largest and the least value scale so far
  float grown = 1.0f;               // 2^-(what the largest one has grown by)

  KeyGroup now[2], next[2];
  uint4 kr[4][2], vr[2][4];
  // table entries are loaded two chunks ahead, scales and codes one
  int ahead[2];
  auto entries = [&](int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = c * kFewKeys + 16 * i;
      ahead[i] = c < c1 && key < hi ? cache_entry(a.pool, b, key >> a.pool.log_bt) : -1;
    }
  };
  auto find = [&](KeyGroup (&kg)[2], int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) kg[i].find(a.pool, ahead[i], h, c * kFewKeys + 16 * i);
  };
  auto load_k = [&](const KeyGroup (&kg)[2]) {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        kr[n][i] = ld_codes_if(a.pool.k + (kg[n >> 1].row + 8 * (n & 1) + g) * a.pool.d + 64 * i + 16 * t,
                               kg[n >> 1].row >= 0 && 4 * i + t < pieces);
  };
  // rows of V past the sequence's end may hold anything: they count as zeros
  auto load_v = [&](const KeyGroup (&kg)[2], int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int slot = 2 * t + (n & 1) + 8 * (n >> 1);
        vr[i][n] = ld_codes_if(a.pool.v + (kg[i].row + slot) * a.pool.d + 16 * g,
                               kg[i].row >= 0 && g < pieces && c * kFewKeys + 16 * i + slot < vis.length);
      }
  };

  int c = c0 + warp;
  entries(c);
  find(now, c);
  entries(c + kFewWarps);
  load_k(now);
  load_v(now, c);
  // One step: the warp's next 32 keys, with the value scales near one another or apart.
  auto step = [&](auto are_apart) {
    constexpr bool kApart = decltype(are_apart)::value;
    find(next, c + kFewWarps);
    entries(c + 2 * kFewWarps);
    // scores
    float z[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) z[n][k] = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t word = w == 0 ? kr[n][i].x : w == 1 ? kr[n][i].y : w == 2 ? kr[n][i].z : kr[n][i].w;
          mma_16816(z[n], qf[4 * i + w], codes_to_half2(word), codes_hi_to_half2(word));
        }
    load_k(next);

    // scale, mask, maximum
    const int key0 = c * kFewKeys;
    const bool whole = key0 >= all_lo && key0 + kFewKeys <= all_hi && now[0].row >= 0 && now[1].row >= 0;
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float sk = scale_value(now[n >> 1].ek);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = key0 + 8 * n + 2 * t + (k & 1);
        z[n][k] *= coef[k >> 1] * sk;
        if (!whole && !(key >= row_lo[k >> 1] && key < row_hi[k >> 1] && now[n >> 1].row >= 0)) z[n][k] = -INFINITY;
        top[k >> 1] = fmaxf(top[k >> 1], z[n][k]);
      }
    }
    float keep[2], use[2];
    if constexpr (!kApart) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        top[k] = fmaxf(m[k], quad_max(top[k]));
        use[k] = top[k] == -INFINITY ? 0.0f : top[k];
        const float f = exp2_fast(m[k] - use[k]);
        m[k] = top[k];
        l[k] *= f;
        keep[k] = f * grown;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x[2], t[2] = {-INFINITY, -INFINITY};  // of the groups: value scale, largest score
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[i] = now[i].ev == kScaleNan ? 0.0f : static_cast<float>(now[i].ev - 127);
#pragma unroll
          for (int j = 0; j < 4; ++j) t[i] = fmaxf(t[i], z[2 * i + (j >> 1)][2 * k + (j & 1)]);
        }
        const float to = fmaxf(m[k], ceilf(quad_max(fmaxf(t[0] + x[0], t[1] + x[1]))));
        const float to_z = fmaxf(mz[k], ceilf(quad_max(fmaxf(t[0], t[1]))));
        const float use = to == -INFINITY ? 0.0f : to, use_z = to_z == -INFINITY ? 0.0f : to_z;
        keep[k] = exp2_fast(m[k] - use);
        m[k] = to;
        l[k] *= exp2_fast(mz[k] - use_z);
        mz[k] = to_z;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float& w = z[j >> 1][2 * k + (j & 1)];
          const bool nan = now[j >> 2].ev == kScaleNan && (whole || w != -INFINITY);
          l[k] += exp2_fast(w - use_z);
          w = nan ? scale_value(kScaleNan) : exp2_fast(w + (x[j >> 2] + kWeightBias - use));
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][2 * k] *= keep[k];
        o[j][2 * k + 1] *= keep[k];
      }
    // weights and values
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float fv = scale_value(max(127 + kWeightBias + now[i].ev - most, 1));
      uint32_t pa[4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if constexpr (!kApart) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float& w = z[2 * i + n][k];
            const float e = exp2_fast(w - use[k >> 1]);
            l[k >> 1] += e;
            w = !whole && w == -INFINITY ? 0.0f : e * fv;  // (a scale that is NaN shows where it is seen)
          }
        }
        pa[2 * n] = pack_pair<__half>(make_float2(z[2 * i + n][0], z[2 * i + n][1]));
        pa[2 * n + 1] = pack_pair<__half>(make_float2(z[2 * i + n][2], z[2 * i + n][3]));
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t q[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) q[n] = w == 0 ? vr[i][n].x : w == 1 ? vr[i][n].y : w == 2 ? vr[i][n].z : vr[i][n].w;
        // bytes of keys 2t and 2t + 1 (2t + 8 and 2t + 9) side by side, per column
        const uint32_t lo01 = __byte_perm(q[0], q[1], 0x5140), hi01 = __byte_perm(q[0], q[1], 0x7362);
        const uint32_t lo89 = __byte_perm(q[2], q[3], 0x5140), hi89 = __byte_perm(q[2], q[3], 0x7362);
        mma_16816(o[4 * w], pa, codes_to_half2(lo01), codes_to_half2(lo89));
        mma_16816(o[4 * w + 1], pa, codes_hi_to_half2(lo01), codes_hi_to_half2(lo89));
        mma_16816(o[4 * w + 2], pa, codes_to_half2(hi01), codes_to_half2(hi89));
        mma_16816(o[4 * w + 3], pa, codes_hi_to_half2(hi01), codes_hi_to_half2(hi89));
      }
    }
    load_v(next, c + kFewWarps);
    now[0] = next[0];
    now[1] = next[1];
  };
  bool apart = false;
  for (; c < c1; c += kFewWarps) {
    int newmost = most;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (now[i].row >= 0 && now[i].ev != kScaleNan) {
        newmost = max(newmost, now[i].ev);
        least = min(least, now[i].ev);
      }
    apart = newmost - least > kFewNear;
    if (apart) break;
    grown = scale_value(max(127 - (newmost - most), 1));
    most = newmost;
    step(std::false_type{});
  }
  if (apart) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      mz[k] = ceilf(m[k]);
      const float f = m[k] == -INFINITY ? 1.0f : exp2_fast(m[k] - mz[k]);
      l[k] *= f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][2 * k] *= f;
        o[j][2 * k + 1] *= f;
      }
      m[k] = mz[k] + static_cast<float>(most - 127);
    }
    for (; c < c1; c += kFewWarps) step(std::true_type{});
  }

  // the warps' parts: element 16 n + j of a row lies at 8 j + n
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    l[k] = quad_sum(l[k]);
    if (t == 0) {
      s_m[warp][g + 8 * k] = apart ? mz[k] : m[k];
      s_x[warp][g + 8 * k] = !apart ? static_cast<float>(most - 127) : mz[k] == -INFINITY ? 0.0f : m[k] - mz[k];
      s_l[warp][g + 8 * k] = l[k];
    }
#pragma unroll
    for (int j = 0; j < 16; ++j)
      *reinterpret_cast<float2*>(&s_o[warp][g + 8 * k][8 * j + 2 * t]) = make_float2(o[j][2 * k], o[j][2 * k + 1]);
  }
  __syncthreads();
  const int n_rows = rows - r0 < kCacheFewRows ? rows - r0 : kCacheFewRows;
  const long long all_rows = static_cast<long long>(a.batch) * a.seq * a.q_heads;
  for (int r = warp; r < n_rows; r += kFewWarps) {
    const int s = (r0 + r) / a.group;
    const int head = h * a.group + (r0 + r) % a.group;
    // sums are in units of 2^s_m, values of 2^(s_m + s_x), s_x whole
    float top = s_m[0][r];
#pragma unroll
    for (int w = 1; w < kFewWarps; ++w) top = fmaxf(top, s_m[w][r]);
    const float base = top == -INFINITY ? 0.0f : top;
    float wt[kFewWarps], total = 0.0f, top_x = -INFINITY;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      total += s_l[w][r] * exp2_fast(s_m[w][r] - base);
      top_x = fmaxf(top_x, s_m[w][r] - base + s_x[w][r]);
    }
    top_x = top_x == -INFINITY ? 0.0f : ceilf(top_x);
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) wt[w] = exp2_fast(s_m[w][r] - base + (s_x[w][r] - top_x));
    const bool none = total == 0.0f || s >= vis.count;  // no key seen, or a row of padding: zeros
    // the warps' values times 2^(top_x - 14) / total, in two factors: the power need not be normal
    const int unit = __float2int_rz(top_x) - kWeightBias, half_unit = unit >> 1;
    const float f1 = none ? 0.0f : scale_value(127 + half_unit) / total, f2 = scale_value(127 + unit - half_unit);
    const long long out_row = (static_cast<long long>(b) * a.seq + s) * a.q_heads + head;
    T* out = static_cast<T*>(a.out.p) + b * a.out.sb + s * a.out.ss + head * a.out.sh;
    for (int col = lane; col < a.pool.d; col += 32) {
      const int at = 8 * (col & 15) + (col >> 4);
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) v += s_o[w][r][at] * wt[w];
      v = none ? 0.0f : v * f1 * f2;
      if (a.splits == 1)
        out[col] = from_f32<T>(v);
      else
        a.part_o[(split * all_rows + out_row) * a.pool.d + col] = v;
    }
    if (lane == 0) {
      const float lse2 = none ? -INFINITY : base + log2f(total);
      if (a.splits > 1)
        a.part_lse[split * all_rows + out_row] = lse2;
      else if (a.lse != nullptr)
        a.lse[out_row] = lse2 * 0.693147180559945309f;
    }
  }
}

// out = sum_i w_i o_i / sum_i w_i, w_i = 2^(lse_i - max): a warp per row. A weight is applied as its
// root twice: by itself it may be less than fp32 holds where its values are so large that they count.
template <typename T>
__global__ void __launch_bounds__(128) cache_attention_join_kernel(const CacheAttentionArgs a) {
  const long long all_rows = static_cast<long long>(a.batch) * a.seq * a.q_heads;
  const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= all_rows) return;
  const int head = static_cast<int>(row % a.q_heads);
  const long long bs = row / a.q_heads;
  const int s = static_cast<int>(bs % a.seq), b = static_cast<int>(bs / a.seq);
  float top = -INFINITY;
  for (int i = lane; i < a.splits; i += 32) top = fmaxf(top, a.part_lse[i * all_rows + row]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float base = top == -INFINITY ? 0.0f : top;
  float total = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = 0; i < a.splits; ++i) {
    const float lse = a.part_lse[i * all_rows + row];
    if (lse == -INFINITY) continue;  // that part saw nothing
    const float root = exp2_fast(0.5f * (lse - base));
    total += root * root;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < a.pool.d) v[j] += root * (root * a.part_o[(i * all_rows + row) * a.pool.d + lane + 32 * j]);
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  T* out = static_cast<T*>(a.out.p) + b * a.out.sb + s * a.out.ss + head * a.out.sh;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (lane + 32 * j < a.pool.d) out[lane + 32 * j] = from_f32<T>(total == 0.0f ? 0.0f : v[j] * inv);
  if (lane == 0 && a.lse != nullptr)
    a.lse[row] = total == 0.0f ? -INFINITY : (base + log2f(total)) * 0.693147180559945309f;
}

template <typename T>
cudaError_t launch_few(const CacheAttentionArgs& a, cudaStream_t s) {
  const long long blocks = static_cast<long long>(a.batch) * a.row_tiles * a.pool.heads * a.splits;
  cache_attention_few_kernel<T><<<static_cast<unsigned>(blocks), kFewWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_join(const CacheAttentionArgs& a, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.batch) * a.seq * a.q_heads;
  cache_attention_join_kernel<T><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attention_few(const CacheAttentionArgs& a, int dtype, cudaStream_t s) {
  return dtype == QKV_CTE_DTYPE_BF16 ? launch_few<__nv_bfloat16>(a, s) : launch_few<__half>(a, s);
}

cudaError_t launch_cache_attention_join(const CacheAttentionArgs& a, int dtype, cudaStream_t s) {
  return dtype == QKV_CTE_DTYPE_BF16 ? launch_join<__nv_bfloat16>(a, s) : launch_join<__half>(a, s);
}

}  // namespace qkvcte

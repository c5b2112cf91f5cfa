// Attention of many queries over the 8-bit cache on the tensor cores.
//
//   z_t = c q . k_t,  p_t = 2^(z_t - m),  o = sum_t p_t v_t / sum_t p_t
// with c = scale log2(e) and a running reference m per row: one pass over the keys, nothing
// of the score matrix leaves the SM.
//
// A CTA owns two tiles of 128 query rows (a row is a token and one of the query heads that
// share the key head) and walks the keys 128 at a time:
//   conversion warps read the codes of K and V, turn them into fp16 (exact: e4m3 is a subset)
//     and store them swizzled for the tensor cores, a tile ahead;
//   one thread issues S = Q K^T (both in shared memory) and O += P V (P in tensor memory);
//   two groups of four softmax warps, a thread per row, take S out of tensor memory, and put
//     P back over it as fp16.
// The two row tiles take turns: while one is in its softmax the tensor cores work on the
// other. Codes cannot feed the tensor cores as they are, because both operands of an 8-bit
// product would have to be 8-bit, and weights and queries rounded to three digits are not
// attention; the conversion is shared by 256 rows.
//
// Scales. A key's block scale multiplies its score in fp32. A value's block scale multiplies
// its weight before the rounding to fp16, relative to the largest value scale so far (an
// exact power of two), 2^7 above: with weights of at most 2^8 (below) that fills fp16's
// range from the top, so 28 binary orders keep their digits.
//
// The reference m follows the maximum lazily: O in tensor memory is rescaled only when the
// maximum has grown by more than 2^8 (or a larger value scale has come), which after the
// first tiles is hardly ever; weights then reach 2^8 instead of 1, which costs nothing.
#include "fp32x2.cuh"
#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

namespace {

constexpr int kTileRows = 128;
constexpr int kTileKeys = 128;
constexpr int kAttnThreads = 512;  // 2 x 4 softmax warps, 4 conversion warps, the issuing warp and three idle
constexpr int kStages = 2;
constexpr int kMetaSlots = 4;
constexpr int kHalfBytes = kTileKeys * 128;       // 128 rows of 64 fp16
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kBias = 7;                          // weights are held 2^7 above their value
constexpr float kGrowth = 8.0f;                   // binary orders the maximum may grow before a rescale
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kSCol = 0, kOCol = 256;        // TMEM columns: S (and P) of both tiles, then O
// Registers per thread and role: 8 x 176 + 4 x 104 + 4 x 56 = 16 x 128, what the launch has.
constexpr int kSoftmaxRegs = 176, kConvertRegs = 104, kIssueRegs = 56;
static_assert(8 * kSoftmaxRegs + 4 * kConvertRegs + 4 * kIssueRegs == 16 * 128, "register split");

// What the softmax warps need to know about a tile of keys, by groups of 16.
struct TileMeta {
  float ck[8];      // key scale (NaN: 255)
  int ev[8];        // exponent of the value scale (of an absent or NaN group: 0)
  uint32_t there;   // groups with a page and tokens
  uint32_t vnan;    // groups whose value scale is NaN
  int top_ev;
  int pad;
};

struct Smem {
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t meta_full[kMetaSlots];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  TileMeta meta[kMetaSlots];
};

constexpr size_t kSmemBytes = 1024 + 2 * kTileBytes + 2 * kStages * kTileBytes + sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// fp16 x fp16 -> fp32, M = 128; B K-major, or N-major (the values: rows of keys, lanes contiguous).
__device__ __forceinline__ uint32_t idesc_f16(int n, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// An N-major operand in 128-byte swizzled rows of 64 lanes: the next 64 lanes are one half
// away (leading byte offset), the next 8 keys 1024 bytes (stride byte offset).
__device__ __forceinline__ uint64_t smem_desc_n_major(uint32_t saddr) {
  uint64_t d = smem_desc_sw128(saddr);
  d |= static_cast<uint64_t>(kHalfBytes >> 4) << 16;
  return d;
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));  // 2 ulp
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint4 ld_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// What a CTA works on; every thread finds the same.
struct Work {
  int split, pair, h, b;

  __device__ __forceinline__ Work(const CacheAttentionArgs& a, long long item) {
    split = static_cast<int>(item % a.splits);
    item /= a.splits;
    pair = a.row_tiles - 1 - static_cast<int>(item % a.row_tiles);  // causal rows with most keys first
    item /= a.row_tiles;
    h = static_cast<int>(item % a.pool.heads);
    b = static_cast<int>(item / a.pool.heads);
  }

  int r0, rows;        // first row; rows of this key head in all
  int key_tile0, n;    // first tile of 128 keys, tiles
  bool two;            // a second row tile

  __device__ __forceinline__ void plan(const CacheAttentionArgs& a, const Visible& v) {
    rows = a.seq * a.group;
    r0 = pair * 2 * kTileRows;
    two = rows - r0 > kTileRows;
    const int s_first = r0 / a.group;
    int s_last = (rows - r0 < 2 * kTileRows ? rows - 1 : r0 + 2 * kTileRows - 1) / a.group;
    if (s_last > v.count - 1) s_last = v.count - 1;
    const int lo = v.lo(a, s_first), hi = s_first > s_last ? 0 : v.hi(a, s_last);
    const int t0 = lo / kTileKeys, t1 = hi > lo ? (hi + kTileKeys - 1) / kTileKeys : t0;
    const int all = t1 - t0;
    key_tile0 = t0 + static_cast<int>(static_cast<long long>(all) * split / a.splits);
    n = t0 + static_cast<int>(static_cast<long long>(all) * (split + 1) / a.splits) - key_tile0;
  }
};

// Every role's waits: bounded, and given up when another role has failed.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Smem* sm, uint32_t* status, uint32_t code) {
  if (mbar_wait_bounded(smem_u32(bar), parity, &sm->abort, kWaitNs)) return true;
  atomicOr(status, code);
  *reinterpret_cast<volatile int*>(&sm->abort) = 1;
  return false;
}

// ---------------------------------------------------------------------------------------
// Conversion: 128 threads; in step i a thread has row 16 i + tid / 8, codes 16 (tid % 8) ...
// ---------------------------------------------------------------------------------------
struct CodeTile {
  uint4 c[8];

  // `limit`: rows from it on are zeros.
  __device__ __forceinline__ void load(const CachePool& p, const uint8_t* codes, int page, int h, int key0, int tid,
                                       int pieces, int limit) {
    const int piece = tid & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int pg = __shfl_sync(0xffffffffu, page, i);
      const int row = 16 * i + (tid >> 3);
      c[i] = make_uint4(0, 0, 0, 0);
      if (pg >= 0 && piece < pieces && row < limit) {
        const int slot = (key0 + row) & ((1 << p.log_bt) - 1);
        const long long at = ((static_cast<long long>(pg) * p.heads + h) << p.log_bt) + slot;
        c[i] = ld_codes(codes + at * p.d + 16 * piece);
      }
    }
  }
  // 16 codes become two 16-byte chunks of a row; which goes first alternates so that eight
  // lanes of a row hit all banks.
  __device__ __forceinline__ void store(uint32_t tile, int tid, int pieces) const {
    const int piece = tid & 7;
    if (piece >= pieces) return;
    const int first = piece >> 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 16 * i + (tid >> 3);
      const uint32_t base = tile + (piece >> 2) * kHalfBytes + row * 128;
      const uint32_t lo[4] = {codes_to_half2(c[i].x), codes_hi_to_half2(c[i].x), codes_to_half2(c[i].y),
                              codes_hi_to_half2(c[i].y)};
      const uint32_t hi[4] = {codes_to_half2(c[i].z), codes_hi_to_half2(c[i].z), codes_to_half2(c[i].w),
                              codes_hi_to_half2(c[i].w)};
      const uint32_t chunk = 2 * (piece & 3);
      const uint32_t at0 = base + (((chunk + first) ^ (row & 7)) << 4);
      const uint32_t at1 = base + (((chunk + 1 - first) ^ (row & 7)) << 4);
      st_shared16(at0, first ? hi[0] : lo[0], first ? hi[1] : lo[1], first ? hi[2] : lo[2], first ? hi[3] : lo[3]);
      st_shared16(at1, first ? lo[0] : hi[0], first ? lo[1] : hi[1], first ? lo[2] : hi[2], first ? lo[3] : hi[3]);
    }
  }
};

__device__ __forceinline__ void convert_role(const CacheAttentionArgs& a, const Work& w, const Visible& vis, Smem* sm,
                                             uint32_t s_k, uint32_t s_v) {
  const int tid = threadIdx.x - 256, lane = tid & 31;
  const int pieces = a.pool.d >> 4;
  if ((a.flags & QKV_CTE_FLAG_TEST_STALL) != 0) return;  // test hook: hand out nothing
  // lane i < 8 keeps the page of a tile's i-th group of 16 keys
  auto find = [&](int j) -> int {
    const int key = (w.key_tile0 + j) * kTileKeys + 16 * lane;
    if (j >= w.n || lane >= 8 || key >= vis.length) return -1;
    return static_cast<int>(cache_page(a.pool, w.b, key >> a.pool.log_bt));
  };
  CodeTile k, v;
  int page = find(0), next = find(1);
  auto limit = [&](int j) { return vis.length - (w.key_tile0 + j) * kTileKeys; };
  k.load(a.pool, a.pool.k, page, w.h, w.key_tile0 * kTileKeys, tid, pieces, kTileKeys);
  v.load(a.pool, a.pool.v, page, w.h, w.key_tile0 * kTileKeys, tid, pieces, limit(0));
  for (int j = 0; j < w.n; ++j) {
    const int st = j & 1;
    const uint32_t ph = (j >> 1) & 1;
    if (!__all_sync(0xffffffffu, wait_for(&sm->k_empty[st], ph ^ 1u, sm, a.status, kErrProducerEmptyWait))) return;
    if (tid < 32) {
      // the slot's last readers have handed in their weights: the issue of the scores that
      // freed this stage came after them
      TileMeta& m = sm->meta[j & (kMetaSlots - 1)];
      int ek = 0, ev = 0;
      if (page >= 0) {
        const size_t at = static_cast<size_t>(page) * a.pool.heads + w.h;
        ek = __ldg(a.pool.k_sf + at);
        ev = __ldg(a.pool.v_sf + at);
      }
      const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
      const uint32_t vnan = __ballot_sync(0xffffffffu, ev == kScaleNan);
      if (ev == kScaleNan) ev = 0;
      const int top = __reduce_max_sync(0xffffffffu, ev);
      if (lane < 8) {
        m.ck[lane] = scale_value(ek);
        m.ev[lane] = ev;
      }
      if (lane == 0) {
        m.there = there;
        m.vnan = vnan;
        m.top_ev = top;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm->meta_full[j & (kMetaSlots - 1)]));
    }
    k.store(s_k + st * kTileBytes, tid, pieces);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm->k_full[st]));
    const int key0 = (w.key_tile0 + j + 1) * kTileKeys;
    k.load(a.pool, a.pool.k, next, w.h, key0, tid, pieces, kTileKeys);
    if (!__all_sync(0xffffffffu, wait_for(&sm->v_empty[st], ph ^ 1u, sm, a.status, kErrProducerEmptyWait))) return;
    v.store(s_v + st * kTileBytes, tid, pieces);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm->v_full[st]));
    v.load(a.pool, a.pool.v, next, w.h, key0, tid, pieces, limit(j + 1));
    page = next;
    next = find(j + 2);
  }
}

// ---------------------------------------------------------------------------------------
// Issue: one thread
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ bool issue_all(const CacheAttentionArgs& a, const Work& w, Smem* sm, uint32_t s_q,
                                          uint32_t s_k, uint32_t s_v, uint32_t tmem) {
  const int tiles = w.two ? 2 : 1;
  const int steps = a.pool.d >> 4;
  const uint32_t id_s = idesc_f16(kTileKeys, false);
  const uint32_t id_o = idesc_f16(a.pool.d > 64 ? 128 : 64, true);
  auto scores = [&](int x, int st) {
    for (int ks = 0; ks < steps; ++ks) {
      const uint32_t off = (ks >> 2) * kHalfBytes + (ks & 3) * 32;
      mma_f16_ss(tmem + kSCol + x * 128, smem_desc_sw128(s_q + x * kTileBytes + off),
                 smem_desc_sw128(s_k + st * kTileBytes + off), id_s, ks > 0 ? 1u : 0u);
    }
    tc_commit(smem_u32(&sm->s_full[x]));
  };
  if (!wait_for(&sm->k_full[0], 0, sm, a.status, kErrMmaFullWait)) return false;
  for (int x = 0; x < tiles; ++x) {
    if (!wait_for(&sm->q_full[x], 0, sm, a.status, kErrMmaFullWait)) return false;
    tc_fence_after();
    scores(x, 0);
  }
  tc_commit(smem_u32(&sm->k_empty[0]));
  for (int j = 0; j < w.n; ++j) {
    const int st = j & 1, st1 = st ^ 1;
    if (!wait_for(&sm->v_full[st], (j >> 1) & 1, sm, a.status, kErrMmaFullWait)) return false;
    for (int x = 0; x < tiles; ++x) {
      if (!wait_for(&sm->p_full[x], j & 1, sm, a.status, kErrMmaTmemEmptyWait)) return false;
      tc_fence_after();
      for (int ks = 0; ks < kTileKeys / 16; ++ks)
        mma_f16_ts(tmem + kOCol + x * 128, tmem + kSCol + x * 128 + 8 * ks,
                   smem_desc_n_major(s_v + st * kTileBytes + ks * 2048), id_o, (j | ks) != 0 ? 1u : 0u);
      if (x == tiles - 1) tc_commit(smem_u32(&sm->v_empty[st]));
      if (j + 1 == w.n) {
        tc_commit(smem_u32(&sm->o_full[x]));
        continue;
      }
      if (x == 0) {
        if (!wait_for(&sm->k_full[st1], ((j + 1) >> 1) & 1, sm, a.status, kErrMmaFullWait)) return false;
        tc_fence_after();
      }
      scores(x, st1);
      if (x == tiles - 1) tc_commit(smem_u32(&sm->k_empty[st1]));
    }
  }
  return true;
}

// ---------------------------------------------------------------------------------------
// Softmax: a thread per row
// ---------------------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void softmax_role(const CacheAttentionArgs& a, const Work& w, const Visible& vis, Smem* sm,
                                             uint32_t s_q, uint32_t tmem, int x) {
  const int row = threadIdx.x & 127;                   // of the tile: also its TMEM lane
  const int r = w.r0 + x * kTileRows + row;
  const int s = r / a.group, head = w.h * a.group + r % a.group;
  const bool inside = r < w.rows;
  const bool live = inside && s < vis.count;
  const int lo = live ? vis.lo(a, s) : 0, hi = live ? vis.hi(a, s) : 0;
  const uint32_t lanes = static_cast<uint32_t>(row & ~31) << 16;
  const uint32_t t_s = tmem + lanes + kSCol + x * 128, t_o = tmem + lanes + kOCol + x * 128;
  const int d = a.pool.d;
  float coef;

  // the row's queries as fp16, swizzled
  {
    const T* p = static_cast<const T*>(a.q.p) + w.b * a.q.sb + s * a.q.ss + head * a.q.sh;
    uint32_t q[64];
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) q[4 * c + i] = 0;
      if (live && 8 * c < d) {
        if (a.wide) {
          const uint4 v = *reinterpret_cast<const uint4*>(p + 8 * c);
          q[4 * c] = v.x, q[4 * c + 1] = v.y, q[4 * c + 2] = v.z, q[4 * c + 3] = v.w;
        } else {
          const uint16_t* e = reinterpret_cast<const uint16_t*>(p + 8 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) q[4 * c + i] = e[2 * i] | static_cast<uint32_t>(e[2 * i + 1]) << 16;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 64; ++i) top = __vmaxu2(top, q[i] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    const int f = query_factor_field(__float_as_uint(unpack_pair<T>(top).x) & 0x7FFFFFFFu);
    const float up = scale_value(f);
    coef = a.scale_log2 * scale_value(254 - f);
    const uint32_t base = s_q + x * kTileBytes + row * 128;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack_pair<T>(q[4 * c + i]);
        h[i] = pack_pair<__half>(make_float2(v.x * up, v.y * up));
      }
      st_shared16(base + (c >> 3) * kHalfBytes + (((c & 7) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
    }
    fence_proxy_async_smem();
    mbar_arrive(smem_u32(&sm->q_full[x]));
  }

  // keys of [all_lo, all_hi) are seen by every live row of the tile
  const int first_row = w.r0 + x * kTileRows;
  const int last_row = w.rows - first_row < kTileRows ? w.rows - 1 : first_row + kTileRows - 1;
  const int s_last = last_row / a.group < vis.count - 1 ? last_row / a.group : vis.count - 1;
  const int all_lo = vis.lo(a, s_last < 0 ? 0 : s_last), all_hi = vis.hi(a, first_row / a.group);

  float m = -INFINITY, l = 0.0f;
  int ref = 1;
  for (int j = 0; j < w.n; ++j) {
    const int slot = j & (kMetaSlots - 1);
    bool ok = wait_for(&sm->meta_full[slot], (j / kMetaSlots) & 1, sm, a.status, kErrEpilogueTmemFullWait);
    ok = ok && wait_for(&sm->s_full[x], j & 1, sm, a.status, kErrEpilogueTmemFullWait);
    if (!__all_sync(0xffffffffu, ok)) return;
    tc_fence_after();
    const TileMeta& meta = sm->meta[slot];
    float z[kTileKeys];
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(t_s + 32 * c, reinterpret_cast<uint32_t*>(z + 32 * c));
    tmem_ld_wait();

    const int key0 = (w.key_tile0 + j) * kTileKeys;
    const bool whole = key0 >= all_lo && key0 + kTileKeys <= all_hi && meta.there == 0xFFu;
    // bit i of word c: key 32 c + i is seen
    uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
    if (!whole) {
      const uint32_t there = meta.there;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int from = lo - key0 - 32 * c, to = hi - key0 - 32 * c;
        uint32_t bits = to <= 0 ? 0u : to >= 32 ? ~0u : (1u << to) - 1u;
        bits &= from <= 0 ? ~0u : from >= 32 ? 0u : ~((1u << from) - 1u);
        if (!(there >> (2 * c) & 1)) bits &= 0xFFFF0000u;
        if (!(there >> (2 * c) & 2)) bits &= 0x0000FFFFu;
        seen[c] = bits;
      }
#pragma unroll
      for (int i = 0; i < kTileKeys; ++i)
        if (!(seen[i >> 5] >> (i & 31) & 1)) z[i] = -INFINITY;
    }
    float c16[8];
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      c16[g] = coef * meta.ck[g];
      float t = max3(z[16 * g], z[16 * g + 1], z[16 * g + 2]);
#pragma unroll
      for (int i = 3; i < 15; i += 2) t = max3(t, z[16 * g + i], z[16 * g + i + 1]);
      t = fmaxf(t, z[16 * g + 15]);
      top = fmaxf(top, t * c16[g]);
    }
    const int top_ev = meta.top_ev;
    if (__any_sync(0xffffffffu, top > m + kGrowth) || top_ev > ref) {
      const float now = fmaxf(m, top);
      const float use = now == -INFINITY ? 0.0f : now;
      const float keep = exp2_fast(m - use);
      const int newref = max(ref, top_ev);
      if (j > 0) {
        const float f = keep * scale_value(max(127 - (newref - ref), 1));
        for (int c = 0; c < (d > 64 ? 8 : 4); ++c) {
          uint32_t o[16];
          tmem_ld_32x32b_x16(t_o + 16 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st_32x32b_x16(t_o + 16 * c, o);
        }
      }
      l *= keep;
      m = now;
      ref = newref;
    }
    const float use = m == -INFINITY ? 0.0f : m;
    const uint32_t vnan = meta.vnan;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t pk[16];
#pragma unroll
      for (int gg = 0; gg < 2; ++gg) {
        const int g = 2 * c + gg;
        const int lf = max(meta.ev[g] - ref + kBias, -40);  // further down fp16 holds nothing
        const float add = static_cast<float>(lf) - use;
        const float2 cc = make_float2(c16[g], c16[g]), aa = make_float2(add, add);
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2 e = ffma2(make_float2(z[16 * g + 2 * i], z[16 * g + 2 * i + 1]), cc, aa);
          e.x = exp2_fast(e.x);
          e.y = exp2_fast(e.y);
          if (!whole) {  // (a scale that is NaN shows where it is seen)
            if (!(seen[c] >> (16 * gg + 2 * i) & 1)) e.x = 0.0f;
            if (!(seen[c] >> (16 * gg + 2 * i + 1) & 1)) e.y = 0.0f;
          }
          sum = fadd2(sum, e);
          if (vnan != 0 && (vnan >> g & 1)) {
            if (seen[c] >> (16 * gg + 2 * i) & 1) e.x = scale_value(kScaleNan);
            if (seen[c] >> (16 * gg + 2 * i + 1) & 1) e.y = scale_value(kScaleNan);
          }
          pk[8 * gg + i] = pack_pair<__half>(e);
        }
        l = fmaf(sum.x + sum.y, scale_value(127 - lf), l);
      }
      tmem_st_32x32b_x16(t_s + 16 * c, pk);
    }
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(smem_u32(&sm->p_full[x]));
  }

  // the row's result
  const long long all_rows = static_cast<long long>(a.batch) * a.seq * a.q_heads;
  const long long out_row = (static_cast<long long>(w.b) * a.seq + s) * a.q_heads + head;
  if (w.n > 0) {
    const bool ok = wait_for(&sm->o_full[x], 0, sm, a.status, kErrEpilogueTmemFullWait);
    if (!__all_sync(0xffffffffu, ok)) return;
    tc_fence_after();
  }
  const bool none = l == 0.0f || !live;  // no key seen, or a row of padding: zeros
  const float f = none ? 0.0f : scale_value(max(ref - kBias, 0)) / l;
  T* out = static_cast<T*>(a.out.p) + w.b * a.out.sb + s * a.out.ss + head * a.out.sh;
  float* part = a.splits > 1 ? a.part_o + (w.split * all_rows + out_row) * d : nullptr;
  for (int c = 0; c < d / 16; ++c) {
    uint32_t o[16];
    if (w.n > 0) {
      tmem_ld_32x32b_x16(t_o + 16 * c, o);
      tmem_ld_wait();
    }
    if (!inside) continue;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = none ? 0.0f : __uint_as_float(o[i]) * f;
    if (part != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(part + 16 * c)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else if (a.wide_out) {
      uint32_t pk[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) pk[i] = pack_pair<T>(make_float2(v[2 * i], v[2 * i + 1]));
      reinterpret_cast<uint4*>(out + 16 * c)[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      reinterpret_cast<uint4*>(out + 16 * c)[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) out[16 * c + i] = from_f32<T>(v[i]);
    }
  }
  if (inside) {
    const float lse2 = none ? -INFINITY : m + log2f(l);
    if (a.splits > 1)
      a.part_lse[w.split * all_rows + out_row] = lse2;
    else if (a.lse != nullptr)
      a.lse[out_row] = lse2 * 0.693147180559945309f;
  }
}

template <typename T>
__global__ void __launch_bounds__(kAttnThreads, 1) cache_attention_kernel(const CacheAttentionArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_q = smem_u32(smem), s_k = s_q + 2 * kTileBytes, s_v = s_k + kStages * kTileBytes;
  Smem* sm = reinterpret_cast<Smem*>(smem + 2 * kTileBytes + 2 * kStages * kTileBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sm->q_full[i]), kTileRows);
      mbar_init(smem_u32(&sm->s_full[i]), 1);
      mbar_init(smem_u32(&sm->p_full[i]), kTileRows);
      mbar_init(smem_u32(&sm->o_full[i]), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&sm->k_full[i]), 4);
      mbar_init(smem_u32(&sm->k_empty[i]), 1);
      mbar_init(smem_u32(&sm->v_full[i]), 4);
      mbar_init(smem_u32(&sm->v_empty[i]), 1);
    }
    for (int i = 0; i < kMetaSlots; ++i) mbar_init(smem_u32(&sm->meta_full[i]), 1);
    mbar_init(smem_u32(&sm->drain), 1);
    sm->abort = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(&sm->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem;

  Work w(a, blockIdx.x);
  const Visible vis(a, w.b);
  w.plan(a, vis);

  if (warp < 8) {
    regs_up<kSoftmaxRegs>();
    const int x = warp >> 2;
    if (x == 0 || w.two) softmax_role<T>(a, w, vis, sm, s_q, tmem, x);
  } else if (warp < 12) {
    regs_down<kConvertRegs>();
    convert_role(a, w, vis, sm, s_k, s_v);
  } else {
    regs_down<kIssueRegs>();
    if (warp == 12 && lane == 0 && w.n > 0 && !issue_all(a, w, sm, s_q, s_k, s_v, tmem)) {
      // what was issued reads shared memory and writes tensor memory: let it end
      tc_commit(smem_u32(&sm->drain));
      if (!mbar_wait_bounded(smem_u32(&sm->drain), 0, nullptr, kWaitNs)) atomicOr(a.status, kErrDrainWait);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T>
cudaError_t launch_tiles(const CacheAttentionArgs& a, cudaStream_t s) {
  auto k = cache_attention_kernel<T>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  const long long blocks = static_cast<long long>(a.batch) * a.row_tiles * a.pool.heads * a.splits;
  k<<<static_cast<unsigned>(blocks), kAttnThreads, kSmemBytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attention_tiles(const CacheAttentionArgs& a, int dtype, cudaStream_t s) {
  return dtype == QKV_CTE_DTYPE_BF16 ? launch_tiles<__nv_bfloat16>(a, s) : launch_tiles<__half>(a, s);
}

}  // namespace qkvcte

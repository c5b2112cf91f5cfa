// Attention of many queries over the 8-bit cache on the tensor cores.
//
//   z_t = c q . k_t,  o = sum_t 2^z_t v_t / sum_t 2^z_t
// with c = scale log2(e) and running references per row: one pass over the keys, nothing of
// the score matrix leaves the SM.
//
// A pair of CTAs owns two tiles of 256 query rows (a row is a token and one of the query heads
// that share the key head), 128 rows of each tile per CTA, and walks the keys 128 at a time:
//   conversion warps read the codes of K and V, turn them into fp16 (exact: e4m3 is a subset)
//     and store them swizzled for the tensor cores, a tile ahead. Each CTA converts half: 64 of
//     the keys of K, half of the lanes of V;
//   one warp of the leading CTA issues S = Q K^T (both in shared memory) and O += P V (P in
//     tensor memory) as M = 256 instructions over the pair, which read each half where it is;
//   two groups of four softmax warps per CTA, a thread per row, take S out of tensor memory,
//     and put P back over it as fp16.
// The two row tiles take turns: while one is in its softmax the tensor cores work on the
// other. Codes cannot feed the tensor cores as they are, because both operands of an 8-bit
// product would have to be 8-bit, and weights and queries rounded to three digits are not
// attention; the conversion is shared by 512 rows.
//
// What bounds it (972 x 4096, 38 heads of 128: 72.5 us, 1.07 PFLOP/s, 0.57 of the measured rate; 4680 x
// 32760, 40 heads 0.53): a tile of 128 keys takes some 4300 clocks for 2048 of products. An
// instruction with A from shared memory takes 86 to 95 clocks instead of 64 by itself, and each
// row tile goes round a chain of softmax (2000), arrival from the other CTA, O += P V and the
// next S. Tried: a CTA by itself (twice the conversion per SM: 700 TFLOP/s), P through shared
// memory so that S is free sooner (870), two softmax threads per row (590, held by the three
// conversion warps that were left room for), one row tile per pair and two blocks per SM (830).
// Short key ranges are bound by what comes before and after: 32760 queries over 128 keys take 378
// us, 11 a pair of blocks, so that over 512 keys (585) more than half is not products.
//
// Scales. A key's block scale multiplies its score in fp32. A value's block scale 2^x_t multiplies
// its weight before the rounding to fp16 (the products take no more digits at this rate; by 2^-11
// at most, an eighth of what a result's rounding to bf16 may cost and as much as one to fp16, and
// it averages out over the keys), so what is rounded is 2^(z_t + x_t - m), with m the row's own
// maximum of z_t + x_t over the keys it sees: neither a key that it does not see nor one whose
// weight makes its large values negligible takes digits from the others. With 2^7 above, the row's
// largest weight is 2^6 or more: down to 2^-20 of it weights keep fp16's digits, and what is 2^-31
// of it is lost.
// The sum of the 2^z_t has a reference n of its own. As long as the value scales met lie within
// 2^60 of one another its terms are the weights without their 2^x_t, one exponential for both,
// and n is m less the first tile's largest x. Beyond (a page of zeros has the least scale there
// is) the terms are taken by themselves, as 2^(z_t - n) (4680 x 32760, 40 heads 3610 us, were it done
// all the time, 3116 otherwise), and both references are whole numbers: a difference of two that are
// large is exact then. (Otherwise m is the maximum itself: a key that is all a row sees has a weight
// of just 2^7, which fp16 holds, and its value comes out as it is.)
//
// m follows its maximum lazily: O in tensor memory is rescaled only when that has grown by more
// than 2^8, which after the first tiles is hardly ever; weights then reach 2^15 instead of 2^7,
// which costs nothing.
#include <type_traits>

#include "fp32x2.cuh"
#include "internal.h"
#include "kv_cache.cuh"
#include "ptx.cuh"
#include "qkv_cte.h"
#include "vec_io.cuh"

namespace qkvcte {

namespace {

constexpr int kTileRows = 128;     // of a row tile, per CTA
constexpr int kTileKeys = 128;
constexpr int kPairRows = kCacheTileRows;
static_assert(kPairRows == 4 * kTileRows, "two CTAs, two row tiles");
constexpr int kAttnThreads = 416;  // 2 x 4 softmax warps, 4 conversion warps, the issuing warp
constexpr int kStages = 2;
constexpr int kMetaSlots = 4;
constexpr int kQHalf = kTileRows * 128;           // 128 rows of 64 fp16
constexpr int kQBytes = 2 * kQHalf;
constexpr int kKHalf = kTileKeys / 2 * 128;       // this CTA's 64 keys, 64 lanes of them
constexpr int kKBytes = 2 * kKHalf;
constexpr int kVBytes = kTileKeys * 128;          // 128 keys, this CTA's lanes of them (64 at most)
constexpr int kBias = 7;                          // weights are held 2^7 above their value
constexpr float kGrowth = 8.0f;                   // binary orders the maximum may grow before a rescale
constexpr int kNear = 60;                         // binary orders of value scales that share an exponential
constexpr uint64_t kWaitNs = 2000000000ull;
// TMEM columns: S (and P) of both tiles, then O. The block has all 512, so they count from 0.
constexpr uint32_t kSCol = 0, kOCol = 256;

// What the softmax warps need to know about a tile of keys, by groups of 16.
struct TileMeta {
  float2 kx[8];     // key scale (NaN: 255), exponent of the value scale (of an absent or NaN group: origin)
  uint32_t there;   // groups with a page and tokens
  uint32_t vnan;    // groups whose value scale is NaN
  float origin;     // exponent of the first tile's largest value scale (0 without one)
  int apart;        // value scales more than 2^60 apart have been met
};
static_assert(sizeof(TileMeta) % 16 == 0, "pairs of kx in one access");

struct alignas(16) Smem {
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t meta_full[kMetaSlots];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  TileMeta meta[kMetaSlots];
};

constexpr size_t kSmemBytes = 1024 + 2 * kQBytes + kStages * (kKBytes + kVBytes) + sizeof(Smem);
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// Issued by one lane of a warp that is together, so that descriptors stay in uniform registers:
// in a branch of one lane every operand is moved there anew (1000 instead of 750 clocks for
// eight instructions of 64).
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on both CTAs' barrier at this offset when that lane's products so far are done.
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// fp16 x fp16 -> fp32, M = 256; B K-major, or N-major (the values: rows of keys, lanes contiguous).
__device__ __forceinline__ uint32_t idesc_f16(int n, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (16u << 24);
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // 2 ulp; below 2^-126 zero (one instruction, not four)
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void ld_global32(uint32_t* w, const void* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// What a pair of CTAs works on; every thread finds the same.
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
    r0 = pair * kPairRows;
    two = rows - r0 > kPairRows / 2;
    const int s_first = r0 / a.group;
    int s_last = (rows - r0 < kPairRows ? rows - 1 : r0 + kPairRows - 1) / a.group;
    if (s_last > v.count - 1) s_last = v.count - 1;
    const int lo = v.lo(a, s_first), hi = s_first > s_last ? 0 : v.hi(a, s_last);
    const int t0 = lo / kTileKeys, t1 = hi > lo ? (hi + kTileKeys - 1) / kTileKeys : t0;
    const int all = t1 - t0;
    key_tile0 = t0 + static_cast<int>(static_cast<long long>(all) * split / a.splits);
    n = t0 + static_cast<int>(static_cast<long long>(all) * (split + 1) / a.splits) - key_tile0;
  }
};

// Every role's waits: bounded, and given up when another role of the CTA has failed. The
// hardware is asked to hold a waiting warp for up to 100 us at a time: warps that poll take
// issue slots from those that work (5050 instead of 4800 clocks a tile of keys).
__device__ __forceinline__ bool try_wait_held(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(100000)
      : "memory");
  return done != 0;
}
// The same for a barrier on which the other CTA arrives: `acquire_pair` has to follow.
__device__ __forceinline__ bool try_wait_held_pair(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(100000)
      : "memory");
  return done != 0;
}
template <bool kPair = false>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, Smem* sm, uint32_t* status, uint32_t code) {
  const uint32_t at = smem_u32(bar);
  auto once = [&]() { return kPair ? try_wait_held_pair(at, parity) : try_wait_held(at, parity); };
  if (once()) return true;
  const uint64_t t0 = globaltimer_ns();
  do {
    if (once()) return true;
  } while (*reinterpret_cast<volatile int*>(&sm->abort) == 0 && globaltimer_ns() - t0 < kWaitNs);
  atomicOr(status, code);
  *reinterpret_cast<volatile int*>(&sm->abort) = 1;
  return false;
}

// Every warp passes here once, when its first loads are on their way: barriers and tensor memory
// of both CTAs are ready behind it.
__device__ __forceinline__ void start_pair() {
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
}

// Arrive on the leading CTA's barrier at this offset, and what the issuing warp does behind its
// wait for it. Release and acquire hold for the pair (the tensor cores read operands where either
// CTA's threads wrote them), but for shared memory alone: tensor memory has fences of its own, and
// nothing else is handed over. A release of all memory waits for the thread's loads in flight as well
// (972 x 4096, 38 heads 88 us, with these 71; at CTA scope, which does not reach the other CTA, 68).
// (What comes the other way are the tensor cores' own arrivals, behind which no thread's writes stand.)
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), 0))
      : "memory");
}
__device__ __forceinline__ void acquire_pair() {
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}

// ---------------------------------------------------------------------------------------
// Conversion: 128 threads with four pieces of 16 codes of K and of V each. Eight lanes that
// store together have the same piece of eight rows, which the swizzle spreads over all banks.
// ---------------------------------------------------------------------------------------
struct CodePieces {
  uint4 c[4];

  // Piece i lies in the page that lane group0 + step i has (-1: zeros), `slot` rows on.
  // `codes`: the pool from this thread's head, row and piece on. Zeros where row + rows i >= limit.
  template <int kRows>
  __device__ __forceinline__ void load(const CachePool& p, const uint8_t* codes, int page, int group0, int row,
                                       int first_slot, int limit) {
    const uint32_t page_bytes = static_cast<uint32_t>(p.heads * p.d) << p.log_bt;  // < 2^30
    const int mask = (1 << p.log_bt) - 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pg = __shfl_sync(0xffffffffu, page, group0 + kRows / 16 * i);
      c[i] = ld_codes_if(codes + static_cast<uint64_t>(static_cast<uint32_t>(pg)) * page_bytes +
                             static_cast<uint32_t>(((first_slot + kRows * i) & mask) * p.d),
                         pg >= 0 && row + kRows * i < limit);
    }
  }
  // To two 16-byte chunks of a row, kRows rows apart.
  template <int kRows>
  __device__ __forceinline__ void store(uint32_t at) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      st_shared16(at + 128 * kRows * i, codes_to_half2(c[i].x), codes_hi_to_half2(c[i].x), codes_to_half2(c[i].y),
                  codes_hi_to_half2(c[i].y));
      st_shared16((at ^ 16) + 128 * kRows * i, codes_to_half2(c[i].z), codes_hi_to_half2(c[i].z),
                  codes_to_half2(c[i].w), codes_hi_to_half2(c[i].w));
    }
  }
};

__device__ __forceinline__ void convert_role(const CacheAttentionArgs& a, const Work& w, const Visible& vis, Smem* sm,
                                             uint32_t s_k, uint32_t s_v, int rank) {
  const int tid = threadIdx.x - 256, lane = tid & 31;
  if ((a.flags & QKV_CTE_FLAG_TEST_STALL) != 0) {  // test hook: hand out nothing
    start_pair();
    return;
  }
  // K: rows krow + 16 i of this CTA's 64 keys, piece kp of 8. V: rows vrow + 32 i of the 128
  // keys, piece vp of this CTA's half of the lanes (of d rounded up to 32). Threads beyond the
  // lanes store zeros where nothing that counts is read.
  const int pieces = a.pool.d >> 4;
  const int krow = (tid & 7) + ((tid >> 2) & 8), kp = ((tid >> 3) & 3) + ((tid >> 4) & 4);
  const int vrow = (tid & 7) + 8 * (tid >> 5), vp = (tid >> 3) & 3;
  const int half = (pieces + 1) >> 1;
  const int vpiece = rank * half + vp;
  const bool k_mine = kp < pieces, v_mine = vp < half && vpiece < pieces;
  const int bt = 1 << a.pool.log_bt;
  const long long head_row = static_cast<long long>(w.h) << a.pool.log_bt;
  const uint8_t* k_codes = a.pool.k + (head_row + (krow & (bt - 1))) * a.pool.d + 16 * kp;
  const uint8_t* v_codes = a.pool.v + (head_row + (vrow & 15)) * a.pool.d + 16 * vpiece;
  const uint32_t k_at = s_k + (kp >> 2) * kKHalf + krow * 128 + (((2 * (kp & 3)) ^ (krow & 7)) << 4);
  const uint32_t v_at = s_v + vrow * 128 + (((2 * vp) ^ (vrow & 7)) << 4);
  const int vgroup = tid >> 6;
  // Lane i < 8 keeps the page of a tile's i-th group of 16 keys. Every load is issued an
  // iteration before its use: table entries two tiles ahead, scales and codes one.
  auto entry = [&](int j) -> int {
    const int key = (w.key_tile0 + j) * kTileKeys + 16 * lane;
    if (j >= w.n || lane >= 8 || key >= vis.length) return -1;
    return cache_entry(a.pool, w.b, key >> a.pool.log_bt);
  };
  auto checked = [&](int e) { return e >= 0 && e < a.pool.pages ? e : -1; };
  int ek = 0, ev = 0, least = kScaleNan, most = -1, origin = 127;
  auto scales = [&](int page) {
    ek = ev = 0;
    if (page >= 0 && tid < 32) {
      const size_t ph = static_cast<size_t>(page) * a.pool.heads + w.h;
      ek = __ldg(a.pool.k_sf + ph);
      ev = __ldg(a.pool.v_sf + ph);
    }
  };
  // keys past the sequence's end may hold anything: as values they count as zeros
  CodePieces k, v;
  auto load_k = [&](int page) { k.load<16>(a.pool, k_codes, page, 4 * rank, krow, 64 * rank, k_mine ? kTileKeys : 0); };
  auto load_v = [&](int page, int j) {
    v.load<32>(a.pool, v_codes, page, vgroup, vrow, 16 * vgroup,
               v_mine ? vis.length - (w.key_tile0 + j) * kTileKeys : 0);
  };
  int page = checked(entry(0)), ahead = entry(1);
  scales(page);
  load_k(page);
  load_v(page, 0);
  start_pair();
  for (int j = 0; j < w.n; ++j) {
    const int st = j & 1;
    const uint32_t ph = (j >> 1) & 1;
    const int next = checked(ahead);
    ahead = entry(j + 2);
    if (!__all_sync(0xffffffffu, wait_for(&sm->k_empty[st], ph ^ 1u, sm, a.status, kErrProducerEmptyWait))) return;
    if (tid < 32) {
      // the slot's last readers (of tile j - 4) have handed in their weights: the scores that freed
      // this stage, of tile j - 2, were issued behind the weights of tile j - 3
      TileMeta& m = sm->meta[j & (kMetaSlots - 1)];
      const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
      const uint32_t vnan = __ballot_sync(0xffffffffu, ev == kScaleNan);
      const bool counts = page >= 0 && ev != kScaleNan;
      least = min(least, __reduce_min_sync(0xffffffffu, counts ? ev : kScaleNan));
      most = max(most, __reduce_max_sync(0xffffffffu, counts ? ev : -1));
      if (j == 0) {
        if (most < 0) most = 127;
        least = min(least, most);
        origin = most;
      }
      if (lane < 8) {
        const int x = counts ? ev : origin;
        m.kx[lane] = make_float2(scale_value(ek), static_cast<float>(x - 127));
      }
      if (lane == 0) {
        m.there = there;
        m.vnan = vnan;
        m.origin = static_cast<float>(origin - 127);
        m.apart = most - least > kNear;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm->meta_full[j & (kMetaSlots - 1)]));
    }
    k.store<16>(k_at + st * kKBytes);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) arrive_leader(&sm->k_full[st]);
    scales(next);
    load_k(next);
    if (!__all_sync(0xffffffffu, wait_for(&sm->v_empty[st], ph ^ 1u, sm, a.status, kErrProducerEmptyWait))) return;
    v.store<32>(v_at + st * kVBytes);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) arrive_leader(&sm->v_full[st]);
    load_v(next, j + 1);
    page = next;
  }
}

// ---------------------------------------------------------------------------------------
// Issue: one warp of the leading CTA
// ---------------------------------------------------------------------------------------
// kSteps: sixteens of lanes. What stands between two instructions is added to their 64 clocks, so a
// product's are one straight line, whatever the head size: nothing is decided within it, and the
// warp is together from its wait (a vote) to its commit, with the same elected lane throughout.
template <int kSteps>
__device__ __forceinline__ bool issue_all(const CacheAttentionArgs& a, const Work& w, Smem* sm, uint32_t s_q,
                                          uint32_t s_k, uint32_t s_v) {
  const int tiles = __shfl_sync(0xffffffffu, w.two ? 2 : 1, 0);
  const int n = __shfl_sync(0xffffffffu, w.n, 0);
  const uint32_t id_s = idesc_f16(kTileKeys, false);
  const uint32_t id_o = idesc_f16((16 * kSteps + 31) & ~31, true);
  const uint64_t q_desc = smem_desc_sw128(s_q), k_desc = smem_desc_sw128(s_k), v_desc = smem_desc_sw128(s_v);
  auto scores = [&](int x, int st) {
    const uint64_t qd = q_desc + (x * kQBytes >> 4), kd = k_desc + (st * kKBytes >> 4);
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
      mma_f16_ss(kSCol + x * 128, qd + (((ks >> 2) * kQHalf + (ks & 3) * 32) >> 4),
                 kd + (((ks >> 2) * kKHalf + (ks & 3) * 32) >> 4), id_s, ks > 0 ? 1u : 0u);
    commit_both(&sm->s_full[x]);
  };
  // (a wait that one lane gives up, all give up)
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
    const bool ok = __all_sync(0xffffffffu, wait_for<true>(bar, parity, sm, a.status, code));
    acquire_pair();
    tc_fence_after();
    return ok;
  };
  if (!wait(&sm->k_full[0], 0, kErrMmaFullWait)) return false;
  for (int x = 0; x < tiles; ++x) {
    if (!wait(&sm->q_full[x], 0, kErrMmaFullWait)) return false;
    scores(x, 0);
  }
  commit_both(&sm->k_empty[0]);
  for (int j = 0; j < n; ++j) {
    const int st = j & 1, st1 = st ^ 1;
    if (!wait(&sm->v_full[st], (j >> 1) & 1, kErrMmaFullWait)) return false;
    for (int x = 0; x < tiles; ++x) {
      if (!wait(&sm->p_full[x], j & 1, kErrMmaTmemEmptyWait)) return false;
      const uint64_t vd = v_desc + (st * kVBytes >> 4);
#pragma unroll
      for (int ks = 0; ks < kTileKeys / 16; ++ks)
        mma_f16_ts(kOCol + x * 128, kSCol + x * 128 + 8 * ks, vd + (ks * 2048 >> 4), id_o,
                   ks > 0 || j > 0 ? 1u : 0u);
      if (x == tiles - 1) commit_both(&sm->v_empty[st]);
      if (j + 1 == n) {
        commit_both(&sm->o_full[x]);
        continue;
      }
      if (x == 0 && !wait(&sm->k_full[st1], ((j + 1) >> 1) & 1, kErrMmaFullWait)) return false;
      scores(x, st1);
      if (x == tiles - 1) commit_both(&sm->k_empty[st1]);
    }
  }
  return true;
}

__device__ __forceinline__ bool issue(const CacheAttentionArgs& a, const Work& w, Smem* sm, uint32_t s_q, uint32_t s_k,
                                      uint32_t s_v) {
  switch (a.pool.d >> 4) {
    case 1: return issue_all<1>(a, w, sm, s_q, s_k, s_v);
    case 2: return issue_all<2>(a, w, sm, s_q, s_k, s_v);
    case 3: return issue_all<3>(a, w, sm, s_q, s_k, s_v);
    case 4: return issue_all<4>(a, w, sm, s_q, s_k, s_v);
    case 5: return issue_all<5>(a, w, sm, s_q, s_k, s_v);
    case 6: return issue_all<6>(a, w, sm, s_q, s_k, s_v);
    case 7: return issue_all<7>(a, w, sm, s_q, s_k, s_v);
    default: return issue_all<8>(a, w, sm, s_q, s_k, s_v);
  }
}

// ---------------------------------------------------------------------------------------
// Softmax: a thread per row
// ---------------------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void softmax_role(const CacheAttentionArgs& a, const Work& w, const Visible& vis, Smem* sm,
                                             uint32_t s_q, int x, int rank) {
  const int row = threadIdx.x & 127;                   // of the tile: also its TMEM lane
  const int first_row = w.r0 + (2 * x + rank) * kTileRows;
  const int r = first_row + row;
  const int s = r / a.group, head = w.h * a.group + r % a.group;
  const bool inside = r < w.rows;
  const bool live = inside && s < vis.count;
  const int lo = live ? vis.lo(a, s) : 0, hi = live ? vis.hi(a, s) : 0;
  const uint32_t lanes = static_cast<uint32_t>(row & ~31) << 16;
  const uint32_t t_s = lanes + kSCol + x * 128, t_o = lanes + kOCol + x * 128;
  const int d = a.pool.d;
  float coef;

  // the row's queries as fp16, swizzled
  {
    const T* p = static_cast<const T*>(a.q.p) + w.b * a.q.sb + s * a.q.ss + head * a.q.sh;
    uint32_t q[64];
    uint32_t top = 0;
    // a lane's row is its own, so an access is a sector of 32 bytes per lane: with 16 bytes each
    // sector is asked for twice (rows off 32-byte boundaries: by elements; 32760 x 512 takes 2440 us
    // then, 585 otherwise)
#pragma unroll
    for (int c = 0; c < 8; ++c) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[8 * c + i] = 0;
      if (live && 16 * c < d) {
        if (a.wide32) {
          ld_global32(q + 8 * c, p + 16 * c);
        } else {
          const uint16_t* e = reinterpret_cast<const uint16_t*>(p + 16 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i) q[8 * c + i] = e[2 * i] | static_cast<uint32_t>(e[2 * i + 1]) << 16;
        }
      }
    }
    start_pair();
#pragma unroll
    for (int i = 0; i < 64; ++i) top = __vmaxu2(top, q[i] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
    top = __float_as_uint(unpack_pair<T>(top).x) & 0x7FFFFFFFu;
    const int f = query_factor_field(top);
    const float up = scale_value(f);
    coef = query_coef(top, f, a.scale_log2);
    const uint32_t base = s_q + x * kQBytes + row * 128;
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 v = unpack_pair<T>(q[4 * c + i]);
        h[i] = pack_pair<__half>(make_float2(v.x * up, v.y * up));
      }
      st_shared16(base + (c >> 3) * kQHalf + (((c & 7) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive_leader(&sm->q_full[x]);
  }

  // keys of [all_lo, all_hi) are seen by every live row of the tile; without a live row it
  // does not matter what the scores are
  const bool dead = first_row >= w.rows || first_row / a.group >= vis.count;
  const int last_row = w.rows - first_row < kTileRows ? w.rows - 1 : first_row + kTileRows - 1;
  const int s_last = last_row / a.group < vis.count - 1 ? last_row / a.group : vis.count - 1;
  const int all_lo = vis.lo(a, s_last < 0 ? 0 : s_last), all_hi = vis.hi(a, first_row / a.group);

  // references of the weights and (where scales lie apart) of the sum, minus infinity before a key
  // is seen; the sum
  float m = -INFINITY, n = -INFINITY, l = 0.0f;
  int j = 0;
  auto scored = [&]() {  // the tile's scores and what goes with its keys are there
    bool ok = wait_for(&sm->meta_full[j & (kMetaSlots - 1)], (j / kMetaSlots) & 1, sm, a.status, kErrEpilogueTmemFullWait);
    ok = ok && wait_for(&sm->s_full[x], j & 1, sm, a.status, kErrEpilogueTmemFullWait);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) tc_fence_after();
    return ok;
  };
  auto weigh = [&](auto are_apart) {  // scores to weights, with the value scales near one another or apart
    constexpr bool kApart = decltype(are_apart)::value;
    const TileMeta& meta = sm->meta[j & (kMetaSlots - 1)];
    const int key0 = (w.key_tile0 + j) * kTileKeys;
    float top = -INFINITY, top_z = -INFINITY;  // the tile's maxima of z + x and, where that is wanted, of z
    // the weights' reference follows the first, and the sum with it unless it has its own
    auto follow = [&]() {
      if (!__any_sync(0xffffffffu, top > m + kGrowth || (kApart && m != ceilf(m)))) return;
      const float now = kApart ? fmaxf(ceilf(m), ceilf(top)) : fmaxf(m, top);
      const float f = exp2_fast(m - (now == -INFINITY ? 0.0f : now));
      m = now;
      if (!kApart) l *= f;
      if (j == 0) return;
      for (int c = 0; c < (d > 64 ? 8 : 4); ++c) {
        uint32_t o[16];
        tmem_ld_32x32b_x16(t_o + 16 * c, o);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tmem_st_32x32b_x16(t_o + 16 * c, o);
      }
    };
    auto follow_sum = [&]() {
      const float now = fmaxf(n, ceilf(top_z)), use = now == -INFINITY ? 0.0f : now;
      l *= exp2_fast(n - use);
      n = now;
      return -use;
    };
    if (dead || (key0 >= all_lo && key0 + kTileKeys <= all_hi && meta.there == 0xFFu && meta.vnan == 0)) {
#pragma unroll 2
      for (int c = 0; c < 4; ++c) {
        float z[32];
        tmem_ld_32x32b_x32(t_s + 32 * c, reinterpret_cast<uint32_t*>(z));
        const float4 kx = *reinterpret_cast<const float4*>(&meta.kx[2 * c]);
        tmem_ld_wait();
        float t[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          t[g] = max3(z[16 * g], z[16 * g + 1], z[16 * g + 2]);
#pragma unroll
          for (int i = 3; i < 15; i += 2) t[g] = max3(t[g], z[16 * g + i], z[16 * g + i + 1]);
          t[g] = fmaxf(t[g], z[16 * g + 15]);
        }
        top = max3(top, fmaf(t[0], coef * kx.x, kx.y), fmaf(t[1], coef * kx.z, kx.w));
        if (kApart) top_z = max3(top_z, t[0] * (coef * kx.x), t[1] * (coef * kx.z));
      }
      follow();
      const float up = kBias - (m == -INFINITY ? 0.0f : m), unit = meta.origin - kBias;
      const float up_n = kApart ? follow_sum() : 0.0f;
#pragma unroll 2
      for (int c = 0; c < 4; ++c) {
        float z[32];
        uint32_t pk[16];
        tmem_ld_32x32b_x32(t_s + 32 * c, reinterpret_cast<uint32_t*>(z));
        const float4 kx = *reinterpret_cast<const float4*>(&meta.kx[2 * c]);
        tmem_ld_wait();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float add = (g == 0 ? kx.y : kx.w) + up, mul = coef * (g == 0 ? kx.x : kx.z);
          const float2 cc = make_float2(mul, mul), aa = make_float2(add, add);
          float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float2 e = ffma2(make_float2(z[16 * g + 2 * i], z[16 * g + 2 * i + 1]), cc, aa);
            e.x = exp2_fast(e.x);
            e.y = exp2_fast(e.y);
            sum = fadd2(sum, e);
            pk[8 * g + i] = pack_pair<__half>(e);
          }
          if constexpr (kApart) {
            const float2 nn = make_float2(up_n, up_n);
            sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 e = ffma2(make_float2(z[16 * g + 2 * i], z[16 * g + 2 * i + 1]), cc, nn);
              e.x = exp2_fast(e.x);
              e.y = exp2_fast(e.y);
              sum = fadd2(sum, e);
            }
            l += sum.x + sum.y;
          } else {
            l = fmaf(sum.x + sum.y, exp2_fast(unit - (g == 0 ? kx.y : kx.w)), l);
          }
        }
        tmem_st_32x32b_x16(t_s + 16 * c, pk);
      }
    } else {
      // Masked, or with a NaN among the value scales: 16 keys at a time, scores read twice.
      // Bit i of `seen`: the row sees key i of the group.
      const uint32_t there = meta.there, vnan = meta.vnan;
      auto seen_bits = [&](int g) {
        const int from = lo - key0 - 16 * g, to = hi - key0 - 16 * g;
        uint32_t bits = to <= 0 ? 0u : to >= 16 ? 0xFFFFu : (1u << to) - 1u;
        bits &= from <= 0 ? 0xFFFFu : from >= 16 ? 0u : ~((1u << from) - 1u);
        return (there >> g & 1) != 0 ? bits : 0u;
      };
#pragma unroll 1
      for (int g = 0; g < 8; ++g) {
        uint32_t z[16];
        tmem_ld_32x32b_x16(t_s + 16 * g, z);
        tmem_ld_wait();
        const uint32_t seen = seen_bits(g);
        float t = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) t = fmaxf(t, (seen >> i & 1) ? __uint_as_float(z[i]) : -INFINITY);
        t *= coef * meta.kx[g].x;
        if (kApart) top_z = fmaxf(top_z, t);
        top = fmaxf(top, t + meta.kx[g].y);
      }
      follow();
      const float up = kBias - (m == -INFINITY ? 0.0f : m), unit = meta.origin - kBias;
      const float up_n = kApart ? follow_sum() : 0.0f;
#pragma unroll 1
      for (int g = 0; g < 8; ++g) {
        uint32_t z[16], pk[8];
        tmem_ld_32x32b_x16(t_s + 16 * g, z);
        tmem_ld_wait();
        const uint32_t seen = seen_bits(g);
        const float add = meta.kx[g].y + up, mul = coef * meta.kx[g].x;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float2 e = make_float2(exp2_fast(fmaf(__uint_as_float(z[2 * i]), mul, add)),
                                 exp2_fast(fmaf(__uint_as_float(z[2 * i + 1]), mul, add)));
          const bool sx = seen >> (2 * i) & 1, sy = seen >> (2 * i + 1) & 1;
          e.x = sx ? e.x : 0.0f;
          e.y = sy ? e.y : 0.0f;
          sum += e.x + e.y;
          if (vnan >> g & 1) {  // shows where it is seen
            if (sx) e.x = scale_value(kScaleNan);
            if (sy) e.y = scale_value(kScaleNan);
          }
          pk[i] = pack_pair<__half>(e);
        }
        tmem_st_32x32b_x8(t_s + 8 * g, pk);
        if constexpr (kApart) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float e = exp2_fast(fmaf(__uint_as_float(z[i]), mul, up_n));
            l += (seen >> i & 1) ? e : 0.0f;
          }
        } else {
          l = fmaf(sum, exp2_fast(unit - meta.kx[g].y), l);
        }
      }
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive_leader(&sm->p_full[x]);
  };
  for (; j < w.n; ++j) {
    if (!scored()) return;
    if (sm->meta[j & (kMetaSlots - 1)].apart != 0) break;
    weigh(std::false_type{});
  }
  const bool apart = j < w.n;
  if (apart) {
    const float up = ceilf(m);
    n = up - sm->meta[j & (kMetaSlots - 1)].origin;
    if (m != -INFINITY) l *= exp2_fast(m - up);
    for (; j < w.n; ++j) {
      if (!scored()) return;
      weigh(std::true_type{});
    }
  }

  // the row's result
  const long long all_rows = static_cast<long long>(a.batch) * a.seq * a.q_heads;
  const long long out_row = (static_cast<long long>(w.b) * a.seq + s) * a.q_heads + head;
  int unit = 0;  // O's less the sum's, binary orders
  if (w.n > 0) {
    const bool ok = wait_for(&sm->o_full[x], 0, sm, a.status, kErrEpilogueTmemFullWait);
    if (!__all_sync(0xffffffffu, ok)) return;
    tc_fence_after();
    const float origin = sm->meta[(w.n - 1) & (kMetaSlots - 1)].origin;
    unit = __float2int_rz(apart ? m - n : origin) - kBias;
    if (!apart) n = m - origin;
  }
  const bool none = l == 0.0f || !live;  // no key seen, or a row of padding: zeros
  // O times 2^unit / l, in two factors: the power need not be normal
  const int half_unit = unit >> 1;
  const float f1 = none ? 0.0f : scale_value(127 + half_unit) / l, f2 = scale_value(127 + unit - half_unit);
  const float2 ff1 = make_float2(f1, f1), ff2 = make_float2(f2, f2);
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
    for (int i = 0; i < 16; i += 2) {
      const float2 x = fmul2(fmul2(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), ff1), ff2);
      v[i] = none ? 0.0f : x.x;
      v[i + 1] = none ? 0.0f : x.y;
    }
    if (part != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<float4*>(part + 16 * c)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else if (a.wide32_out) {
      uint32_t pk[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) pk[i] = pack_pair<T>(make_float2(v[2 * i], v[2 * i + 1]));
      st_global_v8_b32(out + 16 * c, pk);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) out[16 * c + i] = from_f32<T>(v[i]);
    }
  }
  if (inside) {
    const float lse2 = none ? -INFINITY : n + log2f(l);
    if (a.splits > 1)
      a.part_lse[w.split * all_rows + out_row] = lse2;
    else if (a.lse != nullptr)
      a.lse[out_row] = lse2 * 0.693147180559945309f;
  }
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kAttnThreads, 1) cache_attention_kernel(const CacheAttentionArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_q = smem_u32(smem), s_k = s_q + 2 * kQBytes, s_v = s_k + kStages * kKBytes;
  Smem* sm = reinterpret_cast<Smem*>(smem + 2 * kQBytes + kStages * (kKBytes + kVBytes));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int rank = static_cast<int>(cluster_ctarank());

  Work w(a, blockIdx.x >> 1);
  const Visible vis(a, w.b);
  w.plan(a, vis);

  if (warp < 8) {
    const int x = warp >> 2;
    if (x == 0 || w.two)
      softmax_role<T>(a, w, vis, sm, s_q, x, rank);
    else
      start_pair();
  } else if (warp < 12) {
    convert_role(a, w, vis, sm, s_k, s_v, rank);
  } else {
    if ((threadIdx.x & 31) == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&sm->q_full[i]), 8);  // a warp's arrival each: four of either CTA
        mbar_init(smem_u32(&sm->s_full[i]), 1);
        mbar_init(smem_u32(&sm->p_full[i]), 8);
        mbar_init(smem_u32(&sm->o_full[i]), 1);
      }
      for (int i = 0; i < kStages; ++i) {
        mbar_init(smem_u32(&sm->k_full[i]), 8);
        mbar_init(smem_u32(&sm->k_empty[i]), 1);
        mbar_init(smem_u32(&sm->v_full[i]), 8);
        mbar_init(smem_u32(&sm->v_empty[i]), 1);
      }
      for (int i = 0; i < kMetaSlots; ++i) mbar_init(smem_u32(&sm->meta_full[i]), 1);
      mbar_init(smem_u32(&sm->drain), 1);
      sm->abort = 0;
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc_pair(smem_u32(&sm->tmem), 512);
    tmem_relinquish_pair();
    start_pair();
    if (rank == 0 && w.n > 0 && !issue(a, w, sm, s_q, s_k, s_v)) {
      // what was issued reads shared memory and writes tensor memory: let it end
      commit_both(&sm->drain);
      if (!mbar_wait_bounded(smem_u32(&sm->drain), 0, nullptr, kWaitNs)) atomicOr(a.status, kErrDrainWait);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of the pair reads the other's memory any more
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc_pair(sm->tmem, 512);
  }
}

template <typename T>
cudaError_t launch_tiles(const CacheAttentionArgs& a, cudaStream_t s) {
  auto k = cache_attention_kernel<T>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  const long long blocks = 2ll * a.batch * a.row_tiles * a.pool.heads * a.splits;
  k<<<static_cast<unsigned>(blocks), kAttnThreads, kSmemBytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attention_tiles(const CacheAttentionArgs& a, int dtype, cudaStream_t s) {
  return dtype == QKV_CTE_DTYPE_BF16 ? launch_tiles<__nv_bfloat16>(a, s) : launch_tiles<__half>(a, s);
}

}  // namespace qkvcte

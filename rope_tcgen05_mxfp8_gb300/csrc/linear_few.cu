// The product in its channel-major form: 128 output channels take the MMA's M side, a
// tile of tokens its N side, and a cluster splits K and joins its sums on chip.
//
// With few tokens the product reads W once and is bound by that read (and, for the
// smallest calls, by latency). K1's 256-token tiles would leave most SMs idle there: 40
// tiles of 128 channels cover N = 5120. So each tile's K blocks are divided among the 1
// to 8 CTAs of a cluster, every CTA streams its share of W once through a ring of
// 128-byte K blocks, and the partial sums [token][channel] meet in shared memory: CTA r
// of the cluster finishes tokens r, r + S, ... by reading all S parts in order through
// distributed shared memory. There is no workspace and no second launch, and the result
// does not depend on the schedule. W's block scales go straight from w_sf to the layout
// tcgen05.cp wants (a warp gathers one word per channel and K block), so no repack
// kernel runs either. Lanes of the epilogue own channels: consecutive lanes store
// consecutive elements, whatever the alignment of O's rows, which is why rows off 32-byte
// boundaries take this form at any token count.
//
// What bounds it: about 8 us of launch, set-up, joining and storing, then 0.33 us per
// 128-byte K block and CTA whatever the token tile up to 64: the MMAs are too small to
// hide their issue (80 cycles each; 300 more per ring stage for its barriers). The loads
// are not the limit: one token, K = 5120, N = 20480 takes 20.7 us in a captured graph (23.5
// launched one by one) where reading W takes 16.0 at the measured copy rate; N = 5120 with K
// split four ways 9.2 us (12.4; floor 4.0).
//
// The tokens carry no block scales (their scale is the fp32 row scale): their side's
// scale factors are the constant 2^0. Every wait is bounded as in K1.
#include <algorithm>

#include "internal.h"
#include "linear_epilogue.cuh"
#include "ptx.cuh"

namespace qkvcte {

namespace {

constexpr int kFewThreads = 256;  // a load, an MMA and two scale warps; all eight finish
constexpr int kChannels = 128;
constexpr int kFewK = 128;  // K elements (bytes) per ring stage
constexpr int kScaleChunk = 8;  // K blocks whose scales are fetched together (32 bytes of each row of w_sf)
constexpr int kFewScaleBytes = 512;  // 32 rows x 16 bytes: word c of row r is channel 32 c + r
constexpr uint64_t kFewWaitNs = 2000000000ull;
constexpr uint32_t kFewStall = 0x1u;  // QKV_CTE_FLAG_TEST_STALL

template <int NT>
struct FewCfg {
  static constexpr int W_BYTES = kChannels * kFewK;
  static constexpr int A_BYTES = NT * kFewK;
  static constexpr int STAGE_BYTES = W_BYTES + A_BYTES;
  static constexpr int SF_BYTES = 2 * kScaleChunk * kFewScaleBytes;  // two chunks
  // alignment slack, W's and the tokens' block scales, barriers, the tokens' row scales
  static constexpr int FIXED = 1024 + SF_BYTES + kFewScaleBytes + 256 + NT * 4;
  // Half an SM's shared memory, so that two CTAs share it: one's tail overlaps the other's
  // loop. (A ring twice as deep for CTAs alone on their SM was no faster: the loop is not
  // bound by its loads.)
  static constexpr int FIT = (113 * 1024 - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr size_t SMEM = FIXED + static_cast<size_t>(STAGES) * STAGE_BYTES;
  static constexpr int SFA_COL = NT, SFB_COL = NT + 2 * kScaleChunk * 4;  // after two chunks of W's scales
  static constexpr uint32_t TMEM_COLS = NT <= 32 ? 128 : 256;
  static_assert(SFB_COL + 4 <= static_cast<int>(TMEM_COLS) && TMEM_COLS <= 256, "TMEM columns, of two CTAs");
  static_assert(STAGES * STAGE_BYTES >= NT * kChannels * 4, "the partial sums reuse the ring");
  static_assert(STAGES >= 3, "pipeline depth");
};

__device__ __forceinline__ void few_failure(uint32_t* status, volatile int* abort_flag, uint32_t code) {
  atomicOr(status, code);
  *abort_flag = 1;
}

// One word of block scales: K blocks 4 kb .. 4 kb + 3 of a channel (127 past K or N).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* row, bool live, int kb, int k_blocks) {
  if (!live) return 0x7F7F7F7Fu;
  if ((k_blocks & 3) == 0) return __ldg(reinterpret_cast<const uint32_t*>(row) + kb);
  uint32_t w = 0x7F7F7F7Fu;
  for (int j = 0; j < 4; ++j)
    if (4 * kb + j < k_blocks)
      w = (w & ~(0xFFu << (8 * j))) | static_cast<uint32_t>(__ldg(row + 4 * kb + j)) << (8 * j);
  return w;
}

// A thread's two channels, n and n + apart: neighbours where rows keep pairs of elements
// aligned, else 64 apart, so that consecutive lanes store consecutive elements.
struct ChannelParams {
  int n, apart;
  float col[2], bias[2], gate[2];

  __device__ __forceinline__ ChannelParams(const LinearFewArgs& a, int n_, int apart_) : n(n_), apart(apart_) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = n + k * apart;
      const bool in = c < a.N;
      col[k] = a.w_col_scale != nullptr && in ? __ldg(a.w_col_scale + c) : 1.0f;
      bias[k] = a.bias != nullptr && in ? to_f32(reinterpret_cast<const __nv_bfloat16*>(a.bias)[c]) : 0.0f;
      gate[k] = a.lin.gate != nullptr && in ? to_f32(reinterpret_cast<const __nv_bfloat16*>(a.lin.gate)[c]) : 1.0f;
    }
  }
};

template <int kBatch, int kAct, bool kFull>
__device__ __forceinline__ void activate(float2 (&v)[kBatch]) {
#pragma unroll
  for (int u = 0; u < kBatch; ++u) v[u] = make_float2(apply_act<kFull>(v[u].x, kAct), apply_act<kFull>(v[u].y, kAct));
}

// Tokens t, t + step, ... (kBatch of them, those below `live`) of the tile: the sum of
// the cluster's parts in rank order, the epilogue, two elements stored. kMaxParts: the
// cluster's size where it is known, else its largest.
template <int kBatch, int kMaxParts, bool kPairs, typename T>
__device__ __forceinline__ void finish_tokens(const LinearFewArgs& a, const ChannelParams& cp, uint32_t base,
                                              const float* row_scale, int t0, int t, int step, int live) {
  const LinearEpilogue& e = a.lin;
  const int n = cp.n;
  const bool second = n + cp.apart < a.N;
  float2 v[kBatch];
  // the residual as it comes: converting here would wait for each load in turn
  Vec<T, 2> both[kBatch];
  T one[kBatch][2];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int tu = t + u * step;
    v[u] = make_float2(0.0f, 0.0f);
    if (tu < live && e.residual != nullptr) {
      const T* p = static_cast<const T*>(e.residual) + static_cast<long long>(t0 + tu) * e.ldr + n;
      if (kPairs && second) {
        both[u] = *reinterpret_cast<const Vec<T, 2>*>(p);
      } else {
        one[u][0] = p[0];
        if (second) one[u][1] = p[cp.apart];
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int tu = t + u * step;
    if (tu < live) {
      const uint32_t addr = base + 4 * kChannels * tu;
      float2 p[kMaxParts];
#pragma unroll
      for (int r = 0; r < kMaxParts; ++r) {
        p[r] = make_float2(0.0f, 0.0f);
        if constexpr (kMaxParts == 1) {
          p[r] = kPairs ? ld_shared_f32x2(addr) : make_float2(ld_shared_f32(addr), ld_shared_f32(addr + 4 * 64));
        } else if (kMaxParts == 2 || r < a.split) {
          const uint32_t remote = mapa_shared(addr, r);
          p[r] = kPairs ? ld_shared_cluster_f32x2(remote)
                        : make_float2(ld_shared_cluster_f32(remote), ld_shared_cluster_f32(remote + 4 * 64));
        }
      }
      v[u] = p[0];
#pragma unroll
      for (int r = 1; r < kMaxParts; ++r) {
        v[u].x += p[r].x;
        v[u].y += p[r].y;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int tu = t + u * step;
    const float s = row_scale[tu < live ? tu : 0];
    v[u].x = fmaf(v[u].x, s * cp.col[0], cp.bias[0]);
    v[u].y = fmaf(v[u].y, s * cp.col[1], cp.bias[1]);
  }
  constexpr bool kFull = sizeof(T) == 4;
  switch (e.act) {  // one uniform branch for the batch
    case QKV_CTE_ACT_GELU_TANH: activate<kBatch, QKV_CTE_ACT_GELU_TANH, kFull>(v); break;
    case QKV_CTE_ACT_GELU_ERF: activate<kBatch, QKV_CTE_ACT_GELU_ERF, kFull>(v); break;
    case QKV_CTE_ACT_SILU: activate<kBatch, QKV_CTE_ACT_SILU, kFull>(v); break;
    default: break;
  }
  T* out = static_cast<T*>(e.out) + static_cast<long long>(t0 + t) * e.ldo + n;
  const long long pitch = step * e.ldo;
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    if (t + u * step < live) {
      float2 o = make_float2(cp.gate[0] * v[u].x, cp.gate[1] * v[u].y);
      if (e.residual != nullptr) {
        float2 r = make_float2(0.0f, 0.0f);
        if (kPairs && second) {
          r = both[u].pair(0);
        } else {
          r.x = to_f32(one[u][0]);
          if (second) r.y = to_f32(one[u][1]);
        }
        o = make_float2(o.x + r.x, o.y + r.y);
      }
      T* p = out + u * pitch;
      if (kPairs && second) {
        Vec<T, 2> w;
        w.set_pair(0, o);
        st_vec(p, w);
      } else {
        p[0] = from_f32<T>(o.x);
        if (second) p[cp.apart] = from_f32<T>(o.y);
      }
    }
  }
}

// The CTA's tokens rank + split * (group, group + 4, ...), some at a time so that their
// loads overlap.
template <bool kPairs, typename T>
__device__ __forceinline__ void finish_tile(const LinearFewArgs& a, const ChannelParams& cp, uint32_t base,
                                            const float* row_scale, int t0, int rank, int live) {
  const int step = a.split * 4;
  int t = rank + a.split * (static_cast<int>(threadIdx.x) >> 6);
  if (a.split == 1) {
    for (; t < live; t += 8 * step) finish_tokens<8, 1, kPairs, T>(a, cp, base, row_scale, t0, t, step, live);
  } else if (a.split == 2) {
    for (; t < live; t += 8 * step) finish_tokens<8, 2, kPairs, T>(a, cp, base, row_scale, t0, t, step, live);
  } else {
    for (; t < live; t += 2 * step) finish_tokens<2, 8, kPairs, T>(a, cp, base, row_scale, t0, t, step, live);
  }
}

template <int NT>
__global__ void __launch_bounds__(kFewThreads, 2)
    linear_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
                      const LinearFewArgs a) {
  using C = FewCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  constexpr int stages = C::STAGES;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sW = smem;
  uint8_t* sA = sW + stages * C::W_BYTES;
  uint8_t* sSF = sA + stages * C::A_BYTES;
  uint8_t* sOne = sSF + C::SF_BYTES;  // the tokens' scales
  uint64_t* full = reinterpret_cast<uint64_t*>(sOne + kFewScaleBytes);
  uint64_t* empty = full + stages;
  uint64_t* sf_full = empty + stages;  // [2]
  uint64_t* sf_empty = sf_full + 2;     // [2]
  uint64_t* tfull = sf_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * C::STAGES + 5) * 8 + 8 <= 256, "barrier area");
  float* row_scale = reinterpret_cast<float*>(sOne + kFewScaleBytes + 256);  // [NT]
  float* part = reinterpret_cast<float*>(smem);  // [NT][128] once the ring is done

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = a.split;
  const int rank = static_cast<int>(cluster_ctarank());
  const int n0 = (static_cast<int>(blockIdx.x) / split) * kChannels;
  const int t0 = static_cast<int>(blockIdx.y) * NT;
  const int kb0 = static_cast<int>(static_cast<long long>(a.k_stages) * rank / split);
  const int kb1 = static_cast<int>(static_cast<long long>(a.k_stages) * (rank + 1) / split);
  const int n_kb = kb1 - kb0;  // at least one: split <= k_stages

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sf_full[s]), 2);  // the two scale warps
      mbar_init(smem_u32(&sf_empty[s]), 1);
    }
    mbar_init(smem_u32(tfull), 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp >= 4) {
    reinterpret_cast<uint32_t*>(sOne)[threadIdx.x - 128] = 0x7F7F7F7Fu;
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // What the end needs of each thread's two channels is requested now.
  const int live_tokens = a.T - t0 < NT ? a.T - t0 : NT;
  const int ch = (static_cast<int>(threadIdx.x) & 63) * (a.lin.pairs ? 2 : 1);
  const ChannelParams cp(a, n0 + ch, a.lin.pairs ? 1 : 64);

  if (warp == 0) {
    if (lane == 0) {
      // W is read once per token tile; with several tiles the others find it in L2
      const uint64_t pol_w = gridDim.y > 1 ? policy_evict_normal() : policy_evict_first();
      const uint64_t pol_a = policy_evict_last();
      int issued = 0;
      auto load_w = [&](int i, int stage) {
        const uint32_t fb = smem_u32(&full[stage]);
        mbar_arrive_expect_tx(fb, C::STAGE_BYTES);
        tma_load_2d(smem_u32(sW + stage * C::W_BYTES), &tmW, (kb0 + i) * kFewK, n0, fb, pol_w);
      };
      auto load_a = [&](int i, int stage) {
        tma_load_2d(smem_u32(sA + stage * C::A_BYTES), &tmA, (kb0 + i) * kFewK, t0, smem_u32(&full[stage]), pol_a);
      };
      const bool stall = (a.flags & kFewStall) != 0;  // test hook: load nothing
      // W does not depend on the producer step (bf16 or packed rows) this kernel may
      // have been launched beside: the first stages' W goes out before the wait for it.
      const int first = stall ? 0 : (n_kb < stages ? n_kb : stages);
      for (int i = 0; i < first; ++i) load_w(i, i);
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int i = 0; i < first; ++i) load_a(i, i);
      issued = first;
      int stage = first == stages ? 0 : first;
      uint32_t phase = first == stages ? 1 : 0;
      for (int i = first; !stall && i < n_kb; ++i) {
        if (!mbar_wait_bounded(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, kFewWaitNs)) {
          few_failure(a.status, abort_flag, kErrProducerEmptyWait);
          break;
        }
        load_w(i, stage);
        load_a(i, stage);
        ++issued;
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // Without a failure the epilogue's wait covers every copy (the MMAs have read them).
      // After one, stay until the last copies have landed.
      if (*abort_flag) {
        const int pending = issued < stages ? issued : stages;
        for (int i = 0; i < pending; ++i) {
          if (stage == 0) {
            stage = stages - 1;
            phase ^= 1u;
          } else {
            --stage;
          }
          if (!mbar_wait_bounded(smem_u32(&full[stage]), phase, nullptr, kFewWaitNs)) {
            few_failure(a.status, abort_flag, kErrDrainWait);
            break;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_mxf8_e4m3(kChannels, NT);
      const uint32_t sfb = tmem_base + C::SFB_COL;
      tc_copy_32x128b_x4(sfb, smem_desc_plain(smem_u32(sOne)));
      int stage = 0;
      uint32_t phase = 0;
      for (int i = 0; i < n_kb; ++i) {
        const int chunk = i / kScaleChunk, slot = chunk & 1;
        const uint32_t sfa = tmem_base + C::SFA_COL + 4 * (slot * kScaleChunk + i % kScaleChunk);
        if (i % kScaleChunk == 0) {
          // all of a chunk's scales at once, into columns the MMAs in flight do not read
          if (!mbar_wait_bounded(smem_u32(&sf_full[slot]), (chunk >> 1) & 1, abort_flag, kFewWaitNs)) {
            few_failure(a.status, abort_flag, kErrMmaFullWait);
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < kScaleChunk; ++j)
            if (i + j < n_kb)
              tc_copy_32x128b_x4(sfa + 4 * j, smem_desc_plain(smem_u32(sSF + (slot * kScaleChunk + j) * kFewScaleBytes)));
          tc_commit(smem_u32(&sf_empty[slot]));
        }
        if (!mbar_wait_bounded(smem_u32(&full[stage]), phase, abort_flag, kFewWaitNs)) {
          few_failure(a.status, abort_flag, kErrMmaFullWait);
          break;
        }
        tc_fence_after();
        const uint64_t wd = smem_desc_sw128(smem_u32(sW + stage * C::W_BYTES));
        const uint64_t ad = smem_desc_sw128(smem_u32(sA + stage * C::A_BYTES));
#pragma unroll
        for (int k = 0; k < kFewK / 32; ++k)
          mma_mxf8(tmem_base, wd + 2 * k, ad + 2 * k, idesc_with_sf_id(idesc, k, 0), sfa, sfb, (i | k) != 0 ? 1u : 0u);
        tc_commit(smem_u32(&empty[stage]));
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      tc_commit(smem_u32(tfull));  // also on failure: every operation issued above has completed
    }
    __syncwarp();
  } else if (warp < 4) {
    // Block scales: warp 2 gathers the words of channels r and 32 + r (r its lane), warp 3
    // of 64 + r and 96 + r, for kScaleChunk K blocks at a time (beside every ring stage instead:
    // 26.9 us against 23.5 for one token, K = 5120, N = 20480).
    const uint8_t* row[2];
    bool live[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = n0 + 32 * (2 * (warp - 2) + c) + lane;
      live[c] = n < a.N;
      row[c] = a.w_sf + static_cast<size_t>(live[c] ? n : 0) * a.k_blocks;
    }
    for (int chunk = 0; chunk * kScaleChunk < n_kb; ++chunk) {
      uint32_t w[kScaleChunk][2];
#pragma unroll
      for (int j = 0; j < kScaleChunk; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          w[j][c] = scale_word(row[c], live[c] && chunk * kScaleChunk + j < n_kb, kb0 + chunk * kScaleChunk + j, a.k_blocks);
      const int slot = chunk & 1;
      bool ok = mbar_wait_bounded(smem_u32(&sf_empty[slot]), ((chunk >> 1) & 1) ^ 1u, abort_flag, kFewWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) few_failure(a.status, abort_flag, kErrProducerEmptyWait);
        break;
      }
#pragma unroll
      for (int j = 0; j < kScaleChunk; ++j)
        *reinterpret_cast<uint2*>(sSF + (slot * kScaleChunk + j) * kFewScaleBytes + 16 * lane + 8 * (warp - 2)) =
            make_uint2(w[j][0], w[j][1]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sf_full[slot]));
    }
    __syncwarp();
  } else if (warp >= 4) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the row scales of a producer step
    for (int t = static_cast<int>(threadIdx.x) - 128; t < live_tokens; t += 128) row_scale[t] = a.a_scale[t0 + t];
  }
  // ---------------- partial sums to shared memory: all warps, two per lane quarter ----------------
  bool ok = mbar_wait_bounded(smem_u32(tfull), 0, abort_flag, kFewWaitNs);
  ok = __all_sync(0xffffffffu, ok && !*abort_flag);
  if (ok) {
    tc_fence_after();
    const int quarter = warp & 3;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    for (int c = 16 * (warp >> 2); c < live_tokens; c += 32) {
      uint32_t r[16];
      tmem_ld_32x32b_x16(t_lane + c, r);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c + j) * kChannels + quarter * 32 + lane] = __uint_as_float(r[j]);
    }
  } else if (lane == 0) {
    few_failure(a.status, abort_flag, kErrEpilogueTmemFullWait);
  }
  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync();  // every CTA's partial sums are in place
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!*abort_flag && n0 + ch < a.N) {
    const uint32_t base = smem_u32(part) + 4 * ch;
    if (a.lin.dtype == QKV_CTE_DTYPE_BF16)
      a.lin.pairs ? finish_tile<true, __nv_bfloat16>(a, cp, base, row_scale, t0, rank, live_tokens)
                  : finish_tile<false, __nv_bfloat16>(a, cp, base, row_scale, t0, rank, live_tokens);
    else if (a.lin.dtype == QKV_CTE_DTYPE_FP16)
      a.lin.pairs ? finish_tile<true, __half>(a, cp, base, row_scale, t0, rank, live_tokens)
                  : finish_tile<false, __half>(a, cp, base, row_scale, t0, rank, live_tokens);
    else
      a.lin.pairs ? finish_tile<true, float>(a, cp, base, row_scale, t0, rank, live_tokens)
                  : finish_tile<false, float>(a, cp, base, row_scale, t0, rank, live_tokens);
  }
  if (split > 1) cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int NT>
cudaError_t launch_few(const CUtensorMap& tmA, const CUtensorMap& tmW, const LinearFewArgs& a, bool after_producer,
                       cudaStream_t s) {
  using C = FewCfg<NT>;
  auto k = linear_few_kernel<NT>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.N + kChannels - 1) / kChannels * a.split, (a.T + NT - 1) / NT);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after_producer ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, tmA, tmW, a);
}

}  // namespace

cudaError_t launch_linear_few(const CUtensorMap& tmA, const CUtensorMap& tmW, int token_tile, const LinearFewArgs& a,
                              bool after_producer, cudaStream_t s) {
  switch (token_tile) {
    case 16: return launch_few<16>(tmA, tmW, a, after_producer, s);
    case 32: return launch_few<32>(tmA, tmW, a, after_producer, s);
    case 64: return launch_few<64>(tmA, tmW, a, after_producer, s);
    case 128: return launch_few<128>(tmA, tmW, a, after_producer, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qkvcte

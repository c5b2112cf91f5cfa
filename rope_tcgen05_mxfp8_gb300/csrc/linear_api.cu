// C-ABI front end of the product with bias, activation, gate and residual
// (qkv_cte_linear_*, documented in qkv_cte.h): plan, workspace, tensor maps, launches.
#include <climits>
#include <new>

#include "api_common.h"
#include "internal.h"
#include "qkv_cte.h"

using namespace qkvcte;

namespace {

// Workspace (256-byte aligned offsets): [0, 256) the status word and the GEMM's counters
// and stamps at the offsets of internal.h, and a word the scale repack clears in the
// status word's place (a run leaves the status of earlier runs alone); then W's repacked
// scales, the counters K1 expects, and the producer step's codes and row scales.
constexpr size_t kSpareWordOffset = 136;

struct LinearLayout {
  size_t sf_off, ready_off, sm_busy_off, act_off, act_scale_off, total;
};

}  // namespace

struct qkv_cte_linear_plan_s {
  qkv_cte_linear_desc d;
  GemmShape g;
  LinearLayout ws;
  bool few;        // the channel-major form; else K1, but for rows it would store element by element
  int token_tile;  // of the channel-major form
  int split;
};

namespace {

// K1's tile width. A wave of tiles (one per CTA pair, 76 pairs on GB300's 152 SMs) takes
// about 12.5, 13.9 and 15.4 us at K = 5120 for widths 128, 192 and 240, proportional to
// the width plus 350, so the widest tile wins many waves and a narrower one few. us a call
// in a captured graph for 128 / 192 / 240: 1024 x 5120 x 1280 21.2 / 22.6 / 23.3 (one wave
// each), 2048 x 5120 x 5120 67 / 48 / 48 (5, 3 and 3), 4096 x 5120 x 5120 113 / 88 / 78 (9,
// 6, 5). At small K the epilogue bounds a tile, and its time goes by the width as well:
// 32760 x 512 x 5120 201 / 178 / 169, 32760 x 1536 x 1536 94 / 76 / 72 (with GELU tanh 110 /
// 98 / 101), 2048 x 1024 x 5120 25.5 / 23.0 / 24.3, 1024 x 1536 x 1536 14.0 / 15.1 / 15.7.
// Of 13 sizes with K from 512 to 20480, with and without GELU, the choice was the fastest or
// within 4 % of it.
int choose_tile_n(long long m_tiles, long long N) {
  int best = 0;
  long long best_cost = 0;
  for (int t : {240, 192, 128}) {
    const long long waves = (m_tiles * ((N + t - 1) / t) + 75) / 76;
    const long long cost = waves * (t + 350);
    if (best == 0 || cost < best_cost) {
      best = t;
      best_cost = cost;
    }
  }
  return best;
}

// Token tile and K split of the channel-major form, and whether it is the form for a
// problem (its rows' alignment aside). Measured on GB300, us a call in a captured graph (for
// K1 with the scales' repack), K1 against it:
//   T, K, N            K1     token tile / split
//   1, 5120, 5120      62     9.2 (16/4)
//   16, 5120, 20480    114    21.2 (16/1)
//   64, 5120, 20480    43     22.4 (64/1)
//   128, 1024, 5120    12.7   8.6 (64/2)
//   256, 5120, 5120    21.5   18.0 (128/2)
//   128, 5120, 20480   43     27.6 (128/1)
//   512, 1024, 5120    14.1   12.6 (128/1)
//   512, 5120, 5120    23.2   25.7 (128/1)
//   256, 5120, 20480   43     51.2 (128/1, 320 tiles)
// It wins while its tiles fit the SMs about once (two CTAs share an SM, at the expense of
// each other's loads); smaller token tiles add CTAs while there are few. (K1 is slow where
// no tile has more than 16 rows, 53 to 121 us; a ragged last panel of tokens costs it what
// a whole one does: 513, 640 and 768 tokens, 5120 x 20480, 68 to 70.)
bool choose_few(const GemmShape& g, int* token_tile, int* split) {
  const long long channel_tiles = (g.I + 127) / 128;
  int nt = 16;
  while (nt < 64 && nt < g.T) nt *= 2;
  if (channel_tiles * ((g.T + nt - 1) / nt) > 80 && g.T > 64) nt = 128;
  const long long tiles = channel_tiles * ((g.T + nt - 1) / nt);
  int s = 1;
  while (s < 8 && 2 * s <= g.k_stages && tiles * 2 * s <= 192) s *= 2;
  *token_tile = nt;
  *split = s;
  return g.T <= 64 || (tiles <= 160 && (g.T <= 256 || (g.T <= 512 && g.H <= 2048)));
}

size_t out_size(const qkv_cte_linear_desc& d) { return d.out_dtype == QKV_CTE_DTYPE_FP32 ? 4 : 2; }

}  // namespace

extern "C" {

int qkv_cte_linear_plan(qkv_cte_linear_plan_t* out, const qkv_cte_linear_desc* desc, size_t* workspace_bytes) {
  const char* who = "qkv_cte_linear_plan";
  if (out == nullptr || desc == nullptr || workspace_bytes == nullptr)
    return fail(QKV_CTE_ERR_INVALID, "%s: null argument", who);
  *out = nullptr;
  const qkv_cte_linear_desc& d = *desc;
  if (d.tokens < 0) return fail(QKV_CTE_ERR_INVALID, "%s: tokens must be >= 0 (got %lld)", who, (long long)d.tokens);
  if (d.tokens > INT32_MAX - 255)  // rows rounded up to whole tiles stay inside 32 bits
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: more than INT32_MAX - 255 tokens", who);
  if (d.in_features <= 0 || d.out_features <= 0)
    return fail(QKV_CTE_ERR_INVALID, "%s: in_features and out_features must be > 0", who);
  if (d.in_features % 32 != 0)
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: in_features %d is not a multiple of 32", who, d.in_features);
  if (d.in_features > 1 << 30 || d.out_features > 1 << 30) return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: in_features or out_features > 2^30", who);
  if (d.act < QKV_CTE_ACT_NONE || d.act > QKV_CTE_ACT_SILU)
    return fail(QKV_CTE_ERR_INVALID, "%s: unknown activation %d", who, d.act);
  if (d.out_dtype < QKV_CTE_DTYPE_BF16 || d.out_dtype > QKV_CTE_DTYPE_FP32)
    return fail(QKV_CTE_ERR_INVALID, "%s: unknown output type %d", who, d.out_dtype);
  if (d.input_layout != QKV_CTE_INPUT_ROW_FP8 && d.input_layout != QKV_CTE_INPUT_PACKED &&
      d.input_layout != QKV_CTE_INPUT_BF16)
    return fail(QKV_CTE_ERR_INVALID, "%s: unknown input layout %d", who, d.input_layout);
  if ((d.flags & ~QKV_CTE_FLAG_TEST_STALL) != 0) return fail(QKV_CTE_ERR_INVALID, "%s: unknown flags 0x%x", who, d.flags);
  qkv_cte_linear_plan_s* p = new (std::nothrow) qkv_cte_linear_plan_s();
  if (p == nullptr) return fail(QKV_CTE_ERR_INVALID, "out of host memory");
  p->d = d;
  GemmShape& g = p->g;
  g.T = (int)d.tokens;
  g.H = d.in_features;
  g.I = d.out_features;
  g.cta_pair = 1;
  g.blocks128 = (g.T + 127) / 128;
  g.m_tiles = (g.T + 255) / 256;
  g.tile_n = choose_tile_n(g.m_tiles, g.I);
  g.n_tiles = (g.I + g.tile_n - 1) / g.tile_n;
  g.k_stages = (g.H + 127) / 128;  // a short last K block reads zeros past the row's end
  if ((long long)g.m_tiles * g.n_tiles > INT32_MAX) {
    delete p;
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: too many output tiles", who);
  }
  g.sf_chunks = gemm_sf_chunks(g.tile_n);
  g.n_qk_tiles = 0;
  make_bands(g, band_tiles(g));
  p->few = choose_few(g, &p->token_tile, &p->split);
  LinearLayout& w = p->ws;
  w.sf_off = 256;
  w.ready_off = w.sf_off;
  w.sm_busy_off = w.ready_off;
  w.act_off = w.sm_busy_off;
  if (!p->few) {
    w.ready_off = w.sf_off + align_up((size_t)g.n_tiles * g.k_stages * g.sf_chunks * kSfBlockBytesPerChunk, 256);
    w.sm_busy_off = w.ready_off + align_up((size_t)g.blocks128 * sizeof(uint32_t), 256);
    w.act_off = w.sm_busy_off + align_up((size_t)kSmTable * sizeof(uint32_t), 256);
  }
  const bool produced = d.input_layout != QKV_CTE_INPUT_ROW_FP8;
  w.act_scale_off = w.act_off + (produced ? align_up((size_t)g.T * g.H, 256) : 0);
  w.total = w.act_scale_off + (produced ? align_up((size_t)g.T * sizeof(float), 256) : 0);
  *workspace_bytes = w.total;
  *out = p;
  return ok();
}

void qkv_cte_linear_destroy(qkv_cte_linear_plan_t plan) { delete plan; }

int qkv_cte_linear_run(qkv_cte_linear_plan_t plan, const void* A, const float* a_scale, const uint8_t* W,
                       const uint8_t* w_sf, const float* w_col_scale, const uint16_t* bias, const uint16_t* gate,
                       const void* residual, int64_t residual_row_stride, void* O, int64_t out_row_stride,
                       void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "qkv_cte_linear_run";
  if (plan == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null plan", who);
  const qkv_cte_linear_desc& d = plan->d;
  const GemmShape& g = plan->g;
  if (g.T == 0) return ok();
  const bool produced = d.input_layout != QKV_CTE_INPUT_ROW_FP8;
  if (!A || !W || !w_sf || !O || !workspace)
    return fail(QKV_CTE_ERR_INVALID, "%s: A, W, w_sf, O and workspace are required", who);
  if (!produced && !a_scale) return fail(QKV_CTE_ERR_INVALID, "%s: a_scale is required with separate FP8 rows", who);
  if (produced && a_scale)
    return fail(QKV_CTE_ERR_INVALID, "%s: a_scale must be NULL with a packed or bf16 input", who);
  const int64_t T = g.T, N = g.I, e = (int64_t)out_size(d);
  if (T > 1 && (out_row_stride < N || (residual && residual_row_stride < N && residual_row_stride != 0)))
    return fail(QKV_CTE_ERR_INVALID, "%s: a row stride is smaller than out_features", who);
  if (out_row_stride > INT64_MAX / 8 / T || (residual && residual_row_stride > INT64_MAX / 8 / T))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: a row stride overflows", who);
  if (!aligned(A, d.input_layout == QKV_CTE_INPUT_PACKED ? 4 : 16) || !aligned(W, 16))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: A (but for packed rows: 4) and W must be 16-byte aligned", who);
  if (!aligned(a_scale, 4) || !aligned(w_sf, 4) || !aligned(O, e) || !aligned(residual, e))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: a_scale and w_sf must be 4-byte aligned, O and residual to their elements",
                who);
  if (!aligned(w_col_scale, 16) || !aligned(bias, 16) || !aligned(gate, 16))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: w_col_scale, bias and gate must be 16-byte aligned", who);
  if (!aligned(workspace, 256)) return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: workspace must be 256-byte aligned", who);
  if (workspace_bytes < plan->ws.total)
    return fail(QKV_CTE_ERR_INVALID, "%s: workspace of %zu bytes is smaller than the planned %zu", who, workspace_bytes,
                plan->ws.total);
  // O may be the residual itself; it shares no byte with anything else that is read or written.
  const size_t row_bytes = (size_t)(N * e);
  const size_t o_bytes = (size_t)((T - 1) * (T > 1 ? out_row_stride : 0) * e) + row_bytes;
  const size_t r_bytes = residual ? (size_t)((T - 1) * (T > 1 ? residual_row_stride : 0) * e) + row_bytes : 0;
  const size_t a_row = (size_t)g.H * (d.input_layout == QKV_CTE_INPUT_BF16 ? 2 : 1) +
                       (d.input_layout == QKV_CTE_INPUT_PACKED ? 4 : 0);
  const struct {
    const void* p;
    size_t n;
  } in[] = {{A, a_row * (size_t)T},  {a_scale, 4 * (size_t)T},      {W, (size_t)N * g.H},
            {w_sf, (size_t)N * (g.H / 32)}, {w_col_scale, 4 * (size_t)N}, {bias, 2 * (size_t)N},
            {gate, 2 * (size_t)N}};
  for (const auto& b : in)
    if (overlaps(b.p, b.n, O, o_bytes) || overlaps(b.p, b.n, workspace, plan->ws.total))
      return fail(QKV_CTE_ERR_INVALID, "%s: O or the workspace overlaps an input", who);
  if (overlaps(O, o_bytes, workspace, plan->ws.total) || overlaps(residual, r_bytes, workspace, plan->ws.total))
    return fail(QKV_CTE_ERR_INVALID, "%s: the workspace overlaps O or the residual", who);
  const bool in_place = residual == O && (T == 1 || residual_row_stride == out_row_stride);
  if (residual && !in_place &&
      strided_rows_overlap(residual, residual_row_stride * e, O, out_row_stride * e, T, (int64_t)row_bytes))
    return fail(QKV_CTE_ERR_INVALID, "%s: O overlaps the residual without being the same rows", who);

  DeviceInfo dev;
  int rc = check_device(&dev);
  if (rc != QKV_CTE_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint8_t* codes = produced ? ws + plan->ws.act_off : static_cast<const uint8_t*>(A);
  const float* scales = produced ? reinterpret_cast<const float*>(ws + plan->ws.act_scale_off) : a_scale;
  LinearEpilogue lin{};
  lin.act = d.act;
  lin.dtype = d.out_dtype;
  lin.gate = gate;
  lin.residual = residual;
  lin.ldr = T > 1 ? residual_row_stride : 0;
  lin.out = O;
  lin.ldo = T > 1 ? out_row_stride : 0;
  lin.wide = aligned(O, 32) && (lin.ldo * e) % 32 == 0 &&
             (!residual || (aligned(residual, 32) && (lin.ldr * e) % 32 == 0));
  lin.pairs = aligned(O, 2 * e) && lin.ldo % 2 == 0 && (!residual || (aligned(residual, 2 * e) && lin.ldr % 2 == 0));
  // K1 would store rows off 32-byte boundaries element by element, a row of its own for each
  // lane. us a call, K1 so / channel-major / K1 on whole rows of one column more: 2048 x 5120 x
  // 5119 124 / 72 / 49, 4096 x 5120 x 20479 817 / 493 / 264, 32760 x 5120 x 5119 1537 / 822 / 493,
  // 32760 x 512 x 5119 1349 / 328 / 169.
  const bool few = plan->few || (!lin.wide && (g.T + plan->token_tile - 1) / plan->token_tile <= 65535);
  uint8_t* sf_packed = ws + plan->ws.sf_off;
  CUtensorMap tmA, tmW, tmSF;
  rc = encode_operand(&tmA, codes, (uint64_t)g.T, (uint64_t)g.H, few ? (uint32_t)plan->token_tile : 128u, "A");
  if (rc != QKV_CTE_OK) return rc;
  rc = encode_operand(&tmW, W, (uint64_t)g.I, (uint64_t)g.H, few ? 128u : (uint32_t)g.tile_n / 2, "W");
  if (rc != QKV_CTE_OK) return rc;
  if (!few && (rc = encode_scales(&tmSF, sf_packed, g)) != QKV_CTE_OK) return rc;

  cudaError_t err = cudaSuccess;
  if (d.input_layout == QKV_CTE_INPUT_PACKED)
    err = launch_unpack_rows(static_cast<const uint8_t*>(A), g.T, g.H, ws + plan->ws.act_off,
                             reinterpret_cast<float*>(ws + plan->ws.act_scale_off), s, dev.sms);
  else if (d.input_layout == QKV_CTE_INPUT_BF16)
    err = launch_row_quantize(static_cast<const uint16_t*>(A), g.T, g.H, ws + plan->ws.act_off,
                              reinterpret_cast<float*>(ws + plan->ws.act_scale_off), nullptr, s, dev.sms);
  if (err != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "%s: producer launch: %s", who, cudaGetErrorString(err));
  if (few) {
    LinearFewArgs fa{};
    fa.a_scale = scales;
    fa.w_col_scale = w_col_scale;
    fa.bias = bias;
    fa.w_sf = w_sf;
    fa.T = g.T;
    fa.N = g.I;
    fa.k_blocks = g.H / 32;
    fa.k_stages = g.k_stages;
    fa.split = plan->split;
    fa.flags = d.flags;
    fa.status = reinterpret_cast<uint32_t*>(ws);
    fa.lin = lin;
    err = launch_linear_few(tmA, tmW, plan->token_tile, fa, produced, s);
    if (err != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "%s: GEMM launch: %s", who, cudaGetErrorString(err));
    return ok();
  }
  unsigned long long* stamps = reinterpret_cast<unsigned long long*>(ws + kStampOffset);
  uint32_t* ready = reinterpret_cast<uint32_t*>(ws + plan->ws.ready_off);
  uint32_t* sm_busy = reinterpret_cast<uint32_t*>(ws + plan->ws.sm_busy_off);
  err = launch_prep(g, w_sf, sf_packed, nullptr, 0, ready, sm_busy, reinterpret_cast<uint32_t*>(ws + kSpareWordOffset),
                    stamps, reinterpret_cast<uint32_t*>(ws + kTaskCounterOffset), nullptr, 0, s, dev.sms, produced);
  if (err != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "%s: scale repack launch: %s", who, cudaGetErrorString(err));
  GemmArgs a{};
  a.a_scale = scales;
  a.w_col_scale = w_col_scale;
  a.bias = bias;
  a.sf_packed = sf_packed;
  a.ready = ready;
  a.sm_busy = sm_busy;
  a.stamps = stamps;
  a.tile_next = reinterpret_cast<uint32_t*>(ws + kTileCounterOffset);
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.flags = d.flags;
  a.d_head = 16;
  a.lin = lin;
  err = launch_gemm_linear(g, tmA, tmW, tmSF, a, s, dev.sms);
  if (err != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "%s: GEMM launch: %s", who, cudaGetErrorString(err));
  return ok();
}

}  // extern "C"

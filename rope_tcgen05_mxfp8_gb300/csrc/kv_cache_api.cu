// C-ABI front end of the 8-bit key/value cache (qkv_cte_cache_*, documented in qkv_cte.h):
// argument checks, the choice of an attention's form, launches.
#include <algorithm>
#include <climits>
#include <new>

#include "api_common.h"
#include "heads_tensor.h"
#include "kv_cache.h"
#include "qkv_cte.h"

using namespace qkvcte;

struct qkv_cte_cache_plan_s {
  qkv_cte_cache_desc d;
  int log_bt;
  size_t code_bytes, scale_bytes;  // of K, and as many of V
};

namespace {

constexpr int kMaxDHead = 128;
constexpr int kMaxSplits = 64;
// Query rows per key head up to which the form for few queries is taken, in tiles of 16 rows that
// read the keys again (from L2); beyond, pairs of blocks on tcgen05, for which fewer than 256
// rows leave part of every product empty. us a call in a captured graph, few rows' form / tcgen05,
// heads of 128, 40 or 8 key heads:
//         40: over 512   over 4096     4 x 32760     8: over 512   over 4096    32760
//   17    11.4 / 13.8    26.0 / 53.2    550 / 1325   11.4 / 13.7   16.6 / 18.9  37.2 / 62.3
//   32    11.6 / 13.7    27.6 / 54.0    566 / 1325   11.5 / 13.7   16.5 / 18.7  37.4 / 62.5
//   64    13.8 / 13.8    49.3 / 55.8   1046 / 1345   11.6 / 13.7   19.0 / 19.0  56.4 / 62.9
//   96    14.4 / 14.0    55.6 / 58.2   1525 / 1361   11.7 / 13.7   21.3 / 20.2  76.6 / 64.1
//   128   22.7 / 14.3    92.0 / 60.9   1893 / 1377   11.8 / 14.0   23.6 / 20.4   106 / 64.2
constexpr int64_t kFewMaxRows = 64;
// Blocks that run at a time: of the form for few rows two on each of 152 SMs, of the other a pair on
// two SMs. Not the current device's count: the workspace is a function of the sizes alone, asked
// for where there may be no device (with another count the keys are divided less evenly, no more).
constexpr int64_t kFewSlots = 2 * 152, kPairSlots = 152 / 2;
// What a block costs beside its keys, in units of the 17 us that either form's block takes for 1024
// keys of 128 lanes when all run: a pair's start and end 9 us (32760 rows over 128 keys take 11 a
// pair, 2 of them for the keys), a block of the few rows' form 4, the launch that joins 4; partial
// results are written and read at 7.6 TB/s, 1.3e8 bytes in a unit.
constexpr double kPairFixed = 0.5, kFewFixed = 0.25, kJoinFixed = 0.25, kJoinBytes = 1.3e8;
constexpr int64_t kMaxPositions = INT32_MAX - 1024;  // positions and rows rounded up to tiles stay inside 32 bits

size_t elem_size(int dtype) { return dtype == QKV_CTE_DTYPE_FP32 ? 4 : 2; }

// A block of memory of the caller's, for the overlap checks.
struct Block {
  const void* p;
  size_t bytes;
  const char* name;
};

int disjoint(const Block& a, const Block& b, const char* who) {
  if (!overlaps(a.p, a.bytes, b.p, b.bytes)) return QKV_CTE_OK;
  return fail(QKV_CTE_ERR_INVALID, "%s: %s and %s overlap", who, a.name, b.name);
}

// The pool's blocks and the table.
struct PoolBlocks {
  Block b[5];
  int n = 0;
};

int check_pool(qkv_cte_cache_plan_t plan, const qkv_cte_cache_pages* pages, int64_t batch, CachePool* out,
               PoolBlocks* blocks, const char* who) {
  if (plan == nullptr || pages == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null argument", who);
  const qkv_cte_cache_pages& g = *pages;
  if (g.k_codes == nullptr || g.k_sf == nullptr || g.v_codes == nullptr || g.v_sf == nullptr)
    return fail(QKV_CTE_ERR_INVALID, "%s: null codes or scales", who);
  if (!aligned(g.k_codes, 16) || !aligned(g.v_codes, 16))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: the codes must be 16-byte aligned", who);
  if (!aligned(g.table, 4)) return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: table must be 4-byte aligned", who);
  if (g.max_blocks < 1) return fail(QKV_CTE_ERR_INVALID, "%s: max_blocks must be >= 1", who);
  if ((static_cast<int64_t>(g.max_blocks) << plan->log_bt) > kMaxPositions)
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: max_blocks %d are too many positions", who, g.max_blocks);
  if (g.table == nullptr) {
    if (batch > 0 && g.max_blocks > plan->d.pages / batch)
      return fail(QKV_CTE_ERR_INVALID, "%s: without a table %lld sequences of %d pages do not fit the pool's %lld", who,
                  (long long)batch, g.max_blocks, (long long)plan->d.pages);
  } else if (g.table_stride != 0 && g.table_stride < g.max_blocks) {
    return fail(QKV_CTE_ERR_INVALID, "%s: table stride %lld is smaller than max_blocks %d", who,
                (long long)g.table_stride, g.max_blocks);
  } else if (batch > 0 && g.table_stride > INT64_MAX / 8 / batch) {
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: table stride overflows", who);
  }
  blocks->b[0] = {g.k_codes, plan->code_bytes, "the codes of K"};
  blocks->b[1] = {g.v_codes, plan->code_bytes, "the codes of V"};
  blocks->b[2] = {g.k_sf, plan->scale_bytes, "the scales of K"};
  blocks->b[3] = {g.v_sf, plan->scale_bytes, "the scales of V"};
  blocks->n = 4;
  if (g.table != nullptr && batch > 0)
    blocks->b[blocks->n++] = {g.table, 4 * static_cast<size_t>((batch - 1) * g.table_stride + g.max_blocks), "the table"};
  for (int i = 0; i < blocks->n; ++i)
    for (int j = 0; j < i; ++j)
      if (const int rc = disjoint(blocks->b[j], blocks->b[i], who)) return rc;
  *out = CachePool{g.k_codes, g.k_sf,       g.v_codes,           g.v_sf,         g.table,     g.table_stride,
                   plan->d.pages, g.max_blocks, plan->d.n_kv_heads, plan->d.d_head, plan->log_bt};
  return QKV_CTE_OK;
}

int check_counts(int64_t batch, int64_t seq, int64_t heads, const char* who) {
  if (batch < 0 || seq < 0) return fail(QKV_CTE_ERR_INVALID, "%s: batch and seq must be >= 0", who);
  if (batch > INT32_MAX || seq > kMaxPositions || (seq > 0 && batch > kMaxPositions / heads / seq))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: more than INT32_MAX - 1024 rows of heads", who);
  return QKV_CTE_OK;
}

int check_index(const int32_t* p, bool required, const char* name, const char* who) {
  if (p == nullptr && required) return fail(QKV_CTE_ERR_INVALID, "%s: null %s", who, name);
  if (!aligned(p, 4)) return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: %s must be 4-byte aligned", who, name);
  return QKV_CTE_OK;
}

// The stride of a dimension of one element is never followed.
HeadsTensor as_args(const HeadsView& t) {
  return HeadsTensor{const_cast<void*>(t.p), t.batch > 1 ? t.sb : 0, t.seq > 1 ? t.ss : 0, t.heads > 1 ? t.sh : 0};
}

// Whether every row of heads starts on a boundary of `bytes` (16, 32).
bool wide_rows(const HeadsTensor& t, size_t elem, size_t bytes = 16) {
  const int64_t n = static_cast<int64_t>(bytes / elem);
  return aligned(t.p, bytes) && t.sb % n == 0 && t.ss % n == 0 && t.sh % n == 0;
}

// Writing and reading back share all but the direction.
int copy_call(qkv_cte_cache_plan_t plan, const qkv_cte_cache_pages* pages, HeadsView k, HeadsView v, int64_t batch,
              int64_t seq, const int32_t* starts, const int32_t* second, bool read, int32_t dtype, void* stream,
              const char* who) {
  CacheCopyArgs a{};
  PoolBlocks pool;
  int rc = check_pool(plan, pages, batch, &a.pool, &pool, who);
  if (rc != QKV_CTE_OK) return rc;
  if (dtype != QKV_CTE_DTYPE_BF16 && dtype != QKV_CTE_DTYPE_FP16 && dtype != QKV_CTE_DTYPE_FP32)
    return fail(QKV_CTE_ERR_INVALID, "%s: unknown dtype %d", who, dtype);
  const int heads = plan->d.n_kv_heads;
  if ((rc = check_counts(batch, seq, heads, who)) != QKV_CTE_OK) return rc;
  if (batch * seq == 0) return ok();
  if (k.p == nullptr && v.p == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: no k and no v", who);
  if ((rc = check_index(starts, true, "starts", who)) != QKV_CTE_OK) return rc;
  if ((rc = check_index(second, read, read ? "lengths" : "counts", who)) != QKV_CTE_OK) return rc;
  if (!read && pages->table != nullptr && pages->table_stride == 0 && batch > 1)
    return fail(QKV_CTE_ERR_INVALID, "%s: sequences that share one row of the table would write the same pages", who);
  const Block index[2] = {{starts, 4 * static_cast<size_t>(batch), "starts"},
                          {second, 4 * static_cast<size_t>(batch), read ? "lengths" : "counts"}};
  HeadsView* const t[2] = {&k, &v};
  size_t bytes[2] = {0, 0};
  a.wide = 1;
  for (int i = 0; i < 2; ++i) {
    HeadsView& x = *t[i];
    if (x.p == nullptr) continue;
    const char* name = i == 0 ? "k" : "v";
    x.batch = batch, x.seq = seq, x.heads = heads, x.d = plan->d.d_head, x.elem = elem_size(dtype);
    if ((rc = check_heads(x, read, name, who, &bytes[i])) != QKV_CTE_OK) return rc;
    const Block self{x.p, bytes[i], name};
    for (int j = 0; j < pool.n; ++j)
      if ((rc = disjoint(self, pool.b[j], who)) != QKV_CTE_OK) return rc;
    for (const Block& b : index)
      if (read && (rc = disjoint(self, b, who)) != QKV_CTE_OK) return rc;
    (i == 0 ? a.k : a.v) = as_args(x);
    if (!wide_rows(i == 0 ? a.k : a.v, x.elem)) a.wide = 0;
  }
  if (read && k.p != nullptr && v.p != nullptr && heads_overlap(k, bytes[0], v, bytes[1]))
    return fail(QKV_CTE_ERR_INVALID, "%s: k and v overlap", who);
  for (int j = 0; j < 4 && !read; ++j)
    for (const Block& b : index)
      if ((rc = disjoint(pool.b[j], b, who)) != QKV_CTE_OK) return rc;
  const int64_t blocks = ((seq + plan->d.block_tokens - 1) >> plan->log_bt) + 1;
  if (blocks > INT32_MAX / heads / batch)
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: more than INT32_MAX pages and heads", who);
  DeviceInfo dev;
  if ((rc = check_device(&dev)) != QKV_CTE_OK) return rc;
  a.starts = starts;
  a.counts = read ? nullptr : second;
  a.lengths = read ? second : nullptr;
  a.batch = static_cast<int>(batch);
  a.seq = static_cast<int>(seq);
  a.blocks = static_cast<int>(blocks);
  const cudaError_t err = read ? launch_cache_read(a, dtype, static_cast<cudaStream_t>(stream))
                               : launch_cache_write(a, dtype, static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(err));
  return ok();
}

// How an attention call is divided.
struct AttentionShape {
  bool few;
  int row_tiles, splits;
};

AttentionShape attention_shape(const qkv_cte_cache_desc& d, int64_t batch, int64_t seq, int32_t n_q_heads,
                               int64_t max_length) {
  AttentionShape s;
  if (max_length > kMaxPositions) max_length = kMaxPositions;
  const int64_t rows = seq * (n_q_heads / d.n_kv_heads);
  s.few = rows <= kFewMaxRows;
  const int per = s.few ? kCacheFewRows : kCacheTileRows;
  s.row_tiles = static_cast<int>((rows + per - 1) / per);
  const int64_t items = batch * d.n_kv_heads * s.row_tiles;
  // Parts of the keys: the fewest waves of blocks, weighed by what a block costs beside its keys and by
  // the joining. (A window is left out, for the workspace does not depend on it either: rows with one
  // may get more parts than they fill.)
  const int64_t slots = s.few ? kFewSlots : kPairSlots;
  const double fixed = s.few ? kFewFixed : kPairFixed;
  const double traffic = static_cast<double>(batch * seq * n_q_heads) * d.d_head * 8 / kJoinBytes;  // of one part: written, read
  const int64_t most = std::min<int64_t>((max_length + 511) / 512, kMaxSplits);
  double best = 0;
  s.splits = 1;
  for (int64_t k = 1; k <= most; ++k) {
    const double waves = static_cast<double>((items * k + slots - 1) / slots);
    const double cost = waves * (static_cast<double>(max_length) / (1024.0 * k) + fixed) + (k > 1 ? kJoinFixed + traffic * k : 0.0);
    if (k == 1 || cost < best) {
      best = cost;
      s.splits = static_cast<int>(k);
    }
  }
  return s;
}

size_t attention_workspace(const qkv_cte_cache_desc& d, int64_t rows, int splits) {
  return splits > 1 ? static_cast<size_t>(splits) * static_cast<size_t>(rows) * (d.d_head + 1) * sizeof(float) : 0;
}

int check_attention(qkv_cte_cache_plan_t plan, int64_t batch, int64_t seq, int32_t n_q_heads, int64_t max_length,
                    const char* who) {
  if (n_q_heads <= 0 || n_q_heads % plan->d.n_kv_heads != 0)
    return fail(QKV_CTE_ERR_INVALID, "%s: n_q_heads %d is not a multiple of the cache's %d heads", who, n_q_heads,
                plan->d.n_kv_heads);
  if (max_length < 0) return fail(QKV_CTE_ERR_INVALID, "%s: max_length must be >= 0", who);
  return check_counts(batch, seq, n_q_heads, who);
}

}  // namespace

extern "C" {

int qkv_cte_cache_plan(qkv_cte_cache_plan_t* out, const qkv_cte_cache_desc* desc, size_t* code_bytes,
                       size_t* scale_bytes) {
  const char* who = "qkv_cte_cache_plan";
  if (out == nullptr || desc == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null argument", who);
  *out = nullptr;
  const qkv_cte_cache_desc& d = *desc;
  if (d.pages < 1 || d.n_kv_heads < 1 || d.d_head < 1)
    return fail(QKV_CTE_ERR_INVALID, "%s: pages, n_kv_heads and d_head must be > 0", who);
  if (d.flags & ~QKV_CTE_FLAG_TEST_STALL) return fail(QKV_CTE_ERR_INVALID, "%s: unknown flags 0x%x", who, d.flags);
  if (d.d_head % 16 != 0 || d.d_head > kMaxDHead)
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: d_head %d is not a multiple of 16 up to %d", who, d.d_head, kMaxDHead);
  int log_bt = 4;
  while (log_bt < 7 && (1 << log_bt) != d.block_tokens) ++log_bt;
  if ((1 << log_bt) != d.block_tokens)
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: block_tokens %d is not 16, 32, 64 or 128", who, d.block_tokens);
  if (d.pages > INT32_MAX || d.n_kv_heads > 65535)
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: pages > INT32_MAX or n_kv_heads > 65535", who);
  qkv_cte_cache_plan_s* p = new (std::nothrow) qkv_cte_cache_plan_s();
  if (p == nullptr) return fail(QKV_CTE_ERR_INVALID, "out of host memory");
  p->d = d;
  p->log_bt = log_bt;
  p->scale_bytes = static_cast<size_t>(d.pages) * d.n_kv_heads;  // < 2^47
  p->code_bytes = p->scale_bytes * d.block_tokens * d.d_head;     // < 2^61
  if (code_bytes != nullptr) *code_bytes = p->code_bytes;
  if (scale_bytes != nullptr) *scale_bytes = p->scale_bytes;
  *out = p;
  return ok();
}

void qkv_cte_cache_destroy(qkv_cte_cache_plan_t plan) { delete plan; }

int qkv_cte_cache_write(qkv_cte_cache_plan_t plan, const qkv_cte_cache_pages* pages, const void* k,
                        int64_t k_batch_stride, int64_t k_row_stride, int64_t k_head_stride, const void* v,
                        int64_t v_batch_stride, int64_t v_row_stride, int64_t v_head_stride, int64_t batch, int64_t seq,
                        const int32_t* starts, const int32_t* counts, int32_t dtype, void* stream) {
  return copy_call(plan, pages, HeadsView{k, k_batch_stride, k_row_stride, k_head_stride},
                   HeadsView{v, v_batch_stride, v_row_stride, v_head_stride}, batch, seq, starts, counts, false, dtype,
                   stream, "qkv_cte_cache_write");
}

int qkv_cte_cache_read(qkv_cte_cache_plan_t plan, const qkv_cte_cache_pages* pages, void* k, int64_t k_batch_stride,
                       int64_t k_row_stride, int64_t k_head_stride, void* v, int64_t v_batch_stride,
                       int64_t v_row_stride, int64_t v_head_stride, int64_t batch, int64_t seq, const int32_t* starts,
                       const int32_t* lengths, int32_t dtype, void* stream) {
  return copy_call(plan, pages, HeadsView{k, k_batch_stride, k_row_stride, k_head_stride},
                   HeadsView{v, v_batch_stride, v_row_stride, v_head_stride}, batch, seq, starts, lengths, true, dtype,
                   stream, "qkv_cte_cache_read");
}

int qkv_cte_cache_attention_workspace(qkv_cte_cache_plan_t plan, int64_t batch, int64_t seq, int32_t n_q_heads,
                                      int64_t max_length, size_t* bytes) {
  const char* who = "qkv_cte_cache_attention_workspace";
  if (plan == nullptr || bytes == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null argument", who);
  *bytes = 0;
  const int rc = check_attention(plan, batch, seq, n_q_heads, max_length, who);
  if (rc != QKV_CTE_OK) return rc;
  const AttentionShape s = attention_shape(plan->d, batch, seq, n_q_heads, max_length);
  *bytes = attention_workspace(plan->d, batch * seq * n_q_heads, s.splits);
  return ok();
}

int qkv_cte_cache_attention(qkv_cte_cache_plan_t plan, const qkv_cte_cache_pages* pages, const void* q,
                            int64_t q_batch_stride, int64_t q_row_stride, int64_t q_head_stride, void* out,
                            int64_t out_batch_stride, int64_t out_row_stride, int64_t out_head_stride, float* lse,
                            int64_t batch, int64_t seq, int32_t n_q_heads, const int32_t* lengths,
                            const int32_t* counts, int64_t max_length, float scale, int32_t causal, int32_t window,
                            int32_t dtype, void* workspace, size_t workspace_bytes, uint32_t* status, void* stream) {
  const char* who = "qkv_cte_cache_attention";
  CacheAttentionArgs a{};
  PoolBlocks pool;
  int rc = check_pool(plan, pages, batch, &a.pool, &pool, who);
  if (rc != QKV_CTE_OK) return rc;
  if ((rc = check_attention(plan, batch, seq, n_q_heads, max_length, who)) != QKV_CTE_OK) return rc;
  if (dtype == QKV_CTE_DTYPE_FP32)
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: queries are bf16 or fp16", who);
  if (dtype != QKV_CTE_DTYPE_BF16 && dtype != QKV_CTE_DTYPE_FP16)
    return fail(QKV_CTE_ERR_INVALID, "%s: unknown dtype %d", who, dtype);
  if (!(scale > 0.0f) || scale > 1e30f) return fail(QKV_CTE_ERR_INVALID, "%s: scale must be > 0 and finite", who);
  if (causal != 0 && causal != 1) return fail(QKV_CTE_ERR_INVALID, "%s: causal must be 0 or 1", who);
  if (window < 0 || (window > 0 && !causal))
    return fail(QKV_CTE_ERR_INVALID, "%s: a window is >= 0 and goes with causal", who);
  if (batch * seq == 0) return ok();
  if ((rc = check_index(lengths, true, "lengths", who)) != QKV_CTE_OK) return rc;
  if ((rc = check_index(counts, false, "counts", who)) != QKV_CTE_OK) return rc;
  if (status == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null status", who);
  if (!aligned(status, 4) || !aligned(lse, 4))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: status and lse must be 4-byte aligned", who);
  const int64_t rows = batch * seq * n_q_heads;
  const size_t e = elem_size(dtype);
  size_t qn = 0, on = 0;
  const HeadsView vq{q, q_batch_stride, q_row_stride, q_head_stride, batch, seq, n_q_heads, plan->d.d_head, e};
  const HeadsView vo{out, out_batch_stride, out_row_stride, out_head_stride, batch, seq, n_q_heads, plan->d.d_head, e};
  if ((rc = check_heads(vq, false, "q", who, &qn)) != QKV_CTE_OK) return rc;
  if ((rc = check_heads(vo, true, "out", who, &on)) != QKV_CTE_OK) return rc;
  if (heads_overlap(vq, qn, vo, on)) return fail(QKV_CTE_ERR_INVALID, "%s: q and out overlap", who);
  const AttentionShape s = attention_shape(plan->d, batch, seq, n_q_heads, max_length);
  const size_t need = attention_workspace(plan->d, rows, s.splits);
  if (need > 0) {
    if (workspace == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null workspace", who);
    if (!aligned(workspace, 256)) return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: workspace must be 256-byte aligned", who);
    if (workspace_bytes < need)
      return fail(QKV_CTE_ERR_INVALID, "%s: workspace of %zu bytes is smaller than the %zu needed", who,
                  workspace_bytes, need);
  }
  const size_t idx = 4 * static_cast<size_t>(batch);
  const Block outs[4] = {{out, on, "out"},
                         {lse, 4 * static_cast<size_t>(rows), "lse"},
                         {status, 4, "status"},
                         {need > 0 ? workspace : nullptr, need, "the workspace"}};
  const Block ins[3] = {{lengths, idx, "lengths"}, {counts, idx, "counts"}, {q, qn, "q"}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j)
      if ((rc = disjoint(outs[j], outs[i], who)) != QKV_CTE_OK) return rc;
    for (int j = 0; j < pool.n; ++j)
      if ((rc = disjoint(outs[i], pool.b[j], who)) != QKV_CTE_OK) return rc;
    for (int j = 0; j < (i == 0 ? 2 : 3); ++j)  // q and out: above
      if ((rc = disjoint(outs[i], ins[j], who)) != QKV_CTE_OK) return rc;
  }
  if (batch * plan->d.n_kv_heads * s.row_tiles > INT32_MAX / 2 / s.splits)
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: more than INT32_MAX tiles", who);
  DeviceInfo dev;
  if ((rc = check_device(&dev)) != QKV_CTE_OK) return rc;
  a.q = as_args(vq);
  a.out = as_args(vo);
  a.lse = lse;
  a.lengths = lengths;
  a.counts = counts;
  a.batch = static_cast<int>(batch);
  a.seq = static_cast<int>(seq);
  a.q_heads = n_q_heads;
  a.group = n_q_heads / plan->d.n_kv_heads;
  a.row_tiles = s.row_tiles;
  a.splits = s.splits;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.causal = causal;
  a.window = window;
  a.wide = wide_rows(a.q, e);
  a.wide32 = wide_rows(a.q, e, 32);
  a.wide32_out = wide_rows(a.out, e, 32);
  a.status = status;
  a.flags = plan->d.flags;
  if (s.splits > 1) {
    a.part_o = static_cast<float*>(workspace);
    a.part_lse = a.part_o + static_cast<size_t>(s.splits) * rows * plan->d.d_head;
  }
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t err = s.few ? launch_cache_attention_few(a, dtype, cs) : launch_cache_attention_tiles(a, dtype, cs);
  if (err == cudaSuccess && s.splits > 1) err = launch_cache_attention_join(a, dtype, cs);
  if (err != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "%s launch: %s", who, cudaGetErrorString(err));
  return ok();
}

}  // extern "C"

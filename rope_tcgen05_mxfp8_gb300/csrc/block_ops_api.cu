// C-ABI front end of the block operators beside the projection: argument checks and
// launches (the argument lists are documented in qkv_cte.h).
#include <climits>
#include <cmath>
#include <new>

#include "api_common.h"
#include "block_ops.h"
#include "heads_tensor.h"
#include "internal.h"
#include "qkv_cte.h"

using namespace qkvcte;

struct qkv_cte_rope_plan_s {
  qkv_cte_rope_desc d;
  RopePairs pairs;
};

namespace {

size_t elem_size(int dtype) { return dtype == QKV_CTE_DTYPE_FP32 ? 4 : 2; }

bool known_dtype(int dtype) {
  return dtype == QKV_CTE_DTYPE_BF16 || dtype == QKV_CTE_DTYPE_FP16 || dtype == QKV_CTE_DTYPE_FP32;
}

// A strided row block: `rows` rows of `row_bytes` bytes, `stride` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, stride, row_bytes;
  size_t extent() const { return rows > 0 ? (size_t)((rows - 1) * stride + row_bytes) : 0; }
};

bool rows_overlap(const Rows& a, const Rows& b) {
  return strided_rows_overlap(a.p, a.stride, b.p, b.stride, a.rows, a.row_bytes, b.row_bytes);
}

bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && (a.stride == b.stride || a.rows <= 1); }

int check_types(int dtype, int param_dtype, const char* who) {
  if (!known_dtype(dtype)) return fail(QKV_CTE_ERR_INVALID, "%s: unknown dtype %d", who, dtype);
  if (param_dtype != dtype && param_dtype != QKV_CTE_DTYPE_FP32)
    return fail(QKV_CTE_ERR_INVALID, "%s: the parameters have the tensor's type or fp32 (got %d)", who, param_dtype);
  return QKV_CTE_OK;
}

// Rows and columns of a layer norm, and one strided tensor of it.
int check_shape(int64_t rows, int32_t cols, const char* who) {
  if (rows < 0) return fail(QKV_CTE_ERR_INVALID, "%s: rows must be >= 0", who);
  if (cols <= 0) return fail(QKV_CTE_ERR_INVALID, "%s: cols must be > 0", who);
  if (rows > INT32_MAX) return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: rows > INT32_MAX", who);
  if (cols > 1 << 28)  // column indexes and twice them stay well inside 32 bits
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: cols %d > 2^28", who, cols);
  return QKV_CTE_OK;
}

// An input may repeat one row (stride 0); the rows of an output must not overlap.
int check_tensor(const void* p, int64_t stride, int64_t rows, int32_t cols, size_t elem, bool output, const char* name,
                 const char* who) {
  if (p == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null %s", who, name);
  if (!aligned(p, elem)) return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: %s is not aligned to its elements", who, name);
  if (rows > 1 && !(stride >= cols || (stride == 0 && !output)))
    return fail(QKV_CTE_ERR_INVALID, "%s: row stride %lld of %s is smaller than a row of %d", who, (long long)stride,
                name, cols);
  if (stride > INT64_MAX / 8 / (rows > 0 ? rows : 1))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: size of %s overflows", who, name);
  return QKV_CTE_OK;
}

// What the two rope entry points share: counts, positions or grids.
int rope_rows(qkv_cte_rope_plan_t plan, int64_t batch, int64_t seq, const int32_t* positions,
              int64_t pos_batch_stride, const int32_t* grids, RopeArgs* a, size_t* src_bytes, const char* who) {
  if (plan == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null plan", who);
  if (batch < 0 || seq < 0) return fail(QKV_CTE_ERR_INVALID, "%s: batch and seq must be >= 0", who);
  if (batch > INT32_MAX || seq > INT32_MAX || (seq > 0 && batch > INT32_MAX / seq))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: more than INT32_MAX rows", who);
  if (batch * seq > 0) {
    if ((positions == nullptr) == (grids == nullptr))
      return fail(QKV_CTE_ERR_INVALID, "%s: give positions or grids (one of them)", who);
    if (!aligned(positions, 4) || !aligned(grids, 4))
      return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: positions and grids must be 4-byte aligned", who);
    const int64_t one = seq * plan->pairs.n_axes;
    if (positions != nullptr && pos_batch_stride != 0 && pos_batch_stride < one)
      return fail(QKV_CTE_ERR_INVALID, "%s: position batch stride %lld is smaller than one batch of %lld", who,
                  (long long)pos_batch_stride, (long long)one);
    if (pos_batch_stride > INT64_MAX / 8 / batch)
      return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: position batch stride overflows", who);
    *src_bytes = 4 * (size_t)(grids != nullptr ? batch * plan->pairs.n_axes : (batch - 1) * pos_batch_stride + one);
  }
  static_cast<RopePairs&>(*a) = plan->pairs;
  a->batch = (int)batch;
  a->seq = (int)seq;
  a->positions = positions;
  a->pos_batch_stride = positions != nullptr ? pos_batch_stride : 0;
  a->grids = grids;
  return QKV_CTE_OK;
}

}  // namespace

extern "C" {

int qkv_cte_rope_plan(qkv_cte_rope_plan_t* out, const qkv_cte_rope_desc* desc) {
  const char* who = "qkv_cte_rope_plan";
  if (out == nullptr || desc == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null argument", who);
  *out = nullptr;
  const qkv_cte_rope_desc& d = *desc;
  if (d.d_head <= 0 || d.d_head % 2 != 0) return fail(QKV_CTE_ERR_INVALID, "%s: d_head must be even and > 0", who);
  if (d.d_head > 2 * kRopeMaxPairs)
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: d_head %d > %d", who, d.d_head, 2 * kRopeMaxPairs);
  if (d.n_axes < 1 || d.n_axes > kRopeMaxAxes)
    return fail(QKV_CTE_ERR_INVALID, "%s: 1 to %d axes (got %d)", who, kRopeMaxAxes, d.n_axes);
  if (d.spectrum != QKV_CTE_ROPE_PER_AXIS && d.spectrum != QKV_CTE_ROPE_SHARED)
    return fail(QKV_CTE_ERR_INVALID, "%s: unknown spectrum %d", who, d.spectrum);
  if (d.pairing != QKV_CTE_ROPE_ROTATE_HALF && d.pairing != QKV_CTE_ROPE_INTERLEAVED)
    return fail(QKV_CTE_ERR_INVALID, "%s: unknown pairing %d", who, d.pairing);
  if (!(d.theta >= 1.0) || d.theta > 1e30) return fail(QKV_CTE_ERR_INVALID, "%s: theta must be >= 1 and finite", who);
  long long sum = 0;
  for (int i = 0; i < d.n_axes; ++i) {
    if (d.axis_dims[i] <= 0 || d.axis_dims[i] % 2 != 0)
      return fail(QKV_CTE_ERR_INVALID, "%s: axis_dims[%d] must be even and > 0", who, i);
    sum += d.axis_dims[i];
  }
  if (sum != d.d_head)
    return fail(QKV_CTE_ERR_INVALID, "%s: the axes' dims add up to %lld, not to d_head %d", who, sum, d.d_head);
  qkv_cte_rope_plan_s* p = new (std::nothrow) qkv_cte_rope_plan_s();
  if (p == nullptr) return fail(QKV_CTE_ERR_INVALID, "out of host memory");
  p->d = d;
  p->pairs.d = d.d_head;
  p->pairs.n_axes = d.n_axes;
  int pair = 0;
  for (int i = 0; i < d.n_axes; ++i) {
    p->pairs.first_pair[i] = pair;
    for (int j = 0; j < d.axis_dims[i] / 2; ++j, ++pair) {
      const double e = d.spectrum == QKV_CTE_ROPE_PER_AXIS ? 2.0 * j / d.axis_dims[i] : 2.0 * pair / d.d_head;
      const double turns = std::pow(d.theta, -e) / 6.283185307179586476925;  // at most 1 / (2 pi)
      p->pairs.step[pair] = (unsigned long long)std::ldexp(turns, 64);
    }
  }
  *out = p;
  return ok();
}

void qkv_cte_rope_destroy(qkv_cte_rope_plan_t plan) { delete plan; }

int qkv_cte_rope_tables(qkv_cte_rope_plan_t plan, int64_t batch, int64_t seq, const int32_t* positions,
                        int64_t pos_batch_stride, const int32_t* grids, float* cos_table, float* sin_table,
                        void* stream) {
  const char* who = "qkv_cte_rope_tables";
  RopeArgs a{};
  size_t src = 0;
  int rc = rope_rows(plan, batch, seq, positions, pos_batch_stride, grids, &a, &src, who);
  if (rc != QKV_CTE_OK) return rc;
  if (batch * seq == 0) return ok();
  if (cos_table == nullptr || sin_table == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null table", who);
  if (!aligned(cos_table, 16) || !aligned(sin_table, 16))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: the tables must be 16-byte aligned", who);
  const size_t bytes = (size_t)(batch * seq) * (size_t)plan->d.d_head * sizeof(float);
  const void* from = grids != nullptr ? static_cast<const void*>(grids) : positions;
  if (overlaps(cos_table, bytes, sin_table, bytes) || overlaps(cos_table, bytes, from, src) ||
      overlaps(sin_table, bytes, from, src))
    return fail(QKV_CTE_ERR_INVALID, "%s: buffers overlap", who);
  DeviceInfo dev;
  if ((rc = check_device(&dev)) != QKV_CTE_OK) return rc;
  const cudaError_t e = launch_rope_tables(a, cos_table, sin_table, plan->d.pairing == QKV_CTE_ROPE_ROTATE_HALF,
                                           static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "rope tables launch: %s", cudaGetErrorString(e));
  return ok();
}

int qkv_cte_rope_apply(qkv_cte_rope_plan_t plan, const void* x, int64_t x_batch_stride, int64_t x_row_stride,
                       int64_t x_head_stride, void* y, int64_t y_batch_stride, int64_t y_row_stride,
                       int64_t y_head_stride, int64_t batch, int64_t seq, int32_t heads, const int32_t* positions,
                       int64_t pos_batch_stride, const int32_t* grids, int32_t dtype, int32_t inverse, void* stream) {
  const char* who = "qkv_cte_rope_apply";
  RopeArgs a{};
  size_t src = 0;
  int rc = rope_rows(plan, batch, seq, positions, pos_batch_stride, grids, &a, &src, who);
  if (rc != QKV_CTE_OK) return rc;
  if (!known_dtype(dtype)) return fail(QKV_CTE_ERR_INVALID, "%s: unknown dtype %d", who, dtype);
  if (heads < 0) return fail(QKV_CTE_ERR_INVALID, "%s: heads must be >= 0", who);
  if (inverse != 0 && inverse != 1) return fail(QKV_CTE_ERR_INVALID, "%s: inverse must be 0 or 1", who);
  if (heads > 65535 * 8) return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: %d heads", who, heads);
  if (batch * seq * heads == 0) return ok();
  const size_t e = elem_size(dtype);
  size_t xn = 0, yn = 0;
  const HeadsView vx{x, x_batch_stride, x_row_stride, x_head_stride, batch, seq, heads, plan->d.d_head, e};
  const HeadsView vy{y, y_batch_stride, y_row_stride, y_head_stride, batch, seq, heads, plan->d.d_head, e};
  if ((rc = check_heads(vx, false, "x", who, &xn)) != QKV_CTE_OK) return rc;
  if ((rc = check_heads(vy, true, "y", who, &yn)) != QKV_CTE_OK) return rc;
  const bool same = x == y && (batch == 1 || x_batch_stride == y_batch_stride) &&
                    (seq == 1 || x_row_stride == y_row_stride) && (heads == 1 || x_head_stride == y_head_stride);
  if (!same && heads_overlap(vx, xn, vy, yn))
    return fail(QKV_CTE_ERR_INVALID, "%s: x and y overlap without being the same elements", who);
  const void* from = grids != nullptr ? static_cast<const void*>(grids) : positions;
  if (overlaps(y, yn, from, src)) return fail(QKV_CTE_ERR_INVALID, "%s: y overlaps the positions", who);
  DeviceInfo dev;
  if ((rc = check_device(&dev)) != QKV_CTE_OK) return rc;
  a.heads = heads;
  a.x = x;
  a.y = y;
  // the stride of a dimension of one element is never followed
  a.xb = batch > 1 ? x_batch_stride : 0;
  a.xs = seq > 1 ? x_row_stride : 0;
  a.xh = heads > 1 ? x_head_stride : 0;
  a.yb = batch > 1 ? y_batch_stride : 0;
  a.ys = seq > 1 ? y_row_stride : 0;
  a.yh = heads > 1 ? y_head_stride : 0;
  a.inverse = inverse;
  const cudaError_t err = launch_rope_apply(a, dtype, plan->d.pairing == QKV_CTE_ROPE_ROTATE_HALF,
                                            static_cast<cudaStream_t>(stream));
  if (err != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "rope launch: %s", cudaGetErrorString(err));
  return ok();
}

int qkv_cte_layer_norm(const void* x, int64_t x_row_stride, const void* weight, const void* bias, void* y,
                       int64_t y_row_stride, float* mean, float* rstd, int64_t rows, int32_t cols, float eps,
                       int32_t dtype, int32_t param_dtype, void* stream) {
  const char* who = "qkv_cte_layer_norm";
  int rc = check_types(dtype, param_dtype, who);
  if (rc == QKV_CTE_OK) rc = check_shape(rows, cols, who);
  if (rc != QKV_CTE_OK) return rc;
  if (!(eps >= 0.0f) || eps > 1e30f) return fail(QKV_CTE_ERR_INVALID, "%s: eps must be finite and >= 0", who);
  if (rows == 0) return ok();
  const size_t e = elem_size(dtype), pe = elem_size(param_dtype);
  if ((rc = check_tensor(x, x_row_stride, rows, cols, e, false, "x", who)) != QKV_CTE_OK) return rc;
  if ((rc = check_tensor(y, y_row_stride, rows, cols, e, true, "y", who)) != QKV_CTE_OK) return rc;
  if (!aligned(weight, pe) || !aligned(bias, pe) || !aligned(mean, 4) || !aligned(rstd, 4))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: weight, bias, mean and rstd must be aligned to their elements", who);
  const Rows rx{x, rows, x_row_stride * (int64_t)e, (int64_t)cols * (int64_t)e};
  const Rows ry{y, rows, y_row_stride * (int64_t)e, (int64_t)cols * (int64_t)e};
  const size_t stat = (size_t)rows * sizeof(float);
  if (!same_rows(rx, ry) && rows_overlap(rx, ry))
    return fail(QKV_CTE_ERR_INVALID, "%s: x and y overlap without being the same rows", who);
  for (const void* p : {weight, bias})
    if (overlaps(p, cols * pe, y, ry.extent()) || overlaps(p, cols * pe, mean, stat) || overlaps(p, cols * pe, rstd, stat))
      return fail(QKV_CTE_ERR_INVALID, "%s: an output overlaps the parameters", who);
  for (const Rows& r : {rx, ry})
    if (overlaps(r.p, r.extent(), mean, stat) || overlaps(r.p, r.extent(), rstd, stat))
      return fail(QKV_CTE_ERR_INVALID, "%s: the statistics overlap x or y", who);
  if (overlaps(mean, stat, rstd, stat)) return fail(QKV_CTE_ERR_INVALID, "%s: mean and rstd overlap", who);
  DeviceInfo dev;
  if ((rc = check_device(&dev)) != QKV_CTE_OK) return rc;
  const LayerNormArgs a{x, x_row_stride, weight, bias, y, y_row_stride, mean, rstd, rows, cols, eps};
  const cudaError_t err = launch_layer_norm(a, dtype, param_dtype, static_cast<cudaStream_t>(stream), dev.sms);
  if (err != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "layer norm launch: %s", cudaGetErrorString(err));
  return ok();
}

int qkv_cte_layer_norm_backward_workspace(int64_t rows, int32_t cols, size_t* bytes) {
  const char* who = "qkv_cte_layer_norm_backward_workspace";
  if (bytes == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null argument", who);
  *bytes = 0;
  const int rc = check_shape(rows, cols, who);
  if (rc != QKV_CTE_OK) return rc;
  const int64_t parts = rows < kLayerNormMaxParts ? rows : kLayerNormMaxParts;
  *bytes = (size_t)parts * 2 * (size_t)cols * sizeof(float);
  return ok();
}

int qkv_cte_layer_norm_backward(const void* dy, int64_t dy_row_stride, const void* x, int64_t x_row_stride,
                                const void* weight, const float* mean, const float* rstd, void* dx,
                                int64_t dx_row_stride, void* dweight, void* dbias, int64_t rows, int32_t cols,
                                int32_t dtype, int32_t param_dtype, void* workspace, size_t workspace_bytes,
                                void* stream) {
  const char* who = "qkv_cte_layer_norm_backward";
  int rc = check_types(dtype, param_dtype, who);
  if (rc == QKV_CTE_OK) rc = check_shape(rows, cols, who);
  if (rc != QKV_CTE_OK) return rc;
  if (dx == nullptr && dweight == nullptr && dbias == nullptr)
    return fail(QKV_CTE_ERR_INVALID, "%s: no output (dx, dweight and/or dbias)", who);
  const size_t e = elem_size(dtype), pe = elem_size(param_dtype), par = (size_t)cols * pe;
  if (!aligned(weight, pe) || !aligned(dweight, pe) || !aligned(dbias, pe) || !aligned(mean, 4) || !aligned(rstd, 4))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: parameters and statistics must be aligned to their elements", who);
  if (overlaps(dweight, par, dbias, par) || overlaps(weight, par, dweight, par) || overlaps(weight, par, dbias, par))
    return fail(QKV_CTE_ERR_INVALID, "%s: weight, dweight and dbias overlap", who);
  const bool sums = dweight != nullptr || dbias != nullptr;
  size_t need = 0;
  if ((rc = qkv_cte_layer_norm_backward_workspace(rows, cols, &need)) != QKV_CTE_OK) return rc;
  Rows rg{}, rx{}, rd{};
  if (rows > 0) {
    if ((rc = check_tensor(dy, dy_row_stride, rows, cols, e, false, "dy", who)) != QKV_CTE_OK) return rc;
    if ((rc = check_tensor(x, x_row_stride, rows, cols, e, false, "x", who)) != QKV_CTE_OK) return rc;
    if (dx != nullptr &&
        (rc = check_tensor(dx, dx_row_stride, rows, cols, e, true, "dx", who)) != QKV_CTE_OK)
      return rc;
    if (mean == nullptr || rstd == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: mean and rstd are required", who);
    rg = Rows{dy, rows, dy_row_stride * (int64_t)e, (int64_t)par / (int64_t)pe * (int64_t)e};
    rx = Rows{x, rows, x_row_stride * (int64_t)e, rg.row_bytes};
    if (dx != nullptr) rd = Rows{dx, rows, dx_row_stride * (int64_t)e, rg.row_bytes};
    for (const Rows& r : {rg, rx})
      if (dx != nullptr && !same_rows(r, rd) && rows_overlap(r, rd))
        return fail(QKV_CTE_ERR_INVALID, "%s: dx overlaps dy or x without being the same rows", who);
    const size_t stat = (size_t)rows * sizeof(float);
    const void* outs[3] = {dx, dweight, dbias};
    const size_t out_bytes[3] = {rd.extent(), par, par};
    for (int i = 0; i < 3; ++i) {
      if (overlaps(outs[i], out_bytes[i], mean, stat) || overlaps(outs[i], out_bytes[i], rstd, stat) ||
          (i == 0 && overlaps(dx, out_bytes[0], weight, par)))
        return fail(QKV_CTE_ERR_INVALID, "%s: an output overlaps the statistics or the weight", who);
      if (i > 0 && (overlaps(outs[i], par, dy, rg.extent()) || overlaps(outs[i], par, x, rx.extent()) ||
                    overlaps(outs[i], par, dx, rd.extent())))
        return fail(QKV_CTE_ERR_INVALID, "%s: dweight or dbias overlaps dy, x or dx", who);
    }
    if (sums) {
      if (workspace == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: dweight and dbias need a workspace", who);
      if (!aligned(workspace, 256)) return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: workspace must be 256-byte aligned", who);
      if (workspace_bytes < need)
        return fail(QKV_CTE_ERR_INVALID, "%s: workspace of %zu bytes is smaller than the %zu needed", who,
                    workspace_bytes, need);
      if (overlaps(workspace, need, dy, rg.extent()) || overlaps(workspace, need, x, rx.extent()) ||
          overlaps(workspace, need, dx, rd.extent()) || overlaps(workspace, need, dweight, par) ||
          overlaps(workspace, need, dbias, par) || overlaps(workspace, need, weight, par) ||
          overlaps(workspace, need, mean, stat) || overlaps(workspace, need, rstd, stat))
        return fail(QKV_CTE_ERR_INVALID, "%s: the workspace overlaps a tensor", who);
    }
  }
  if (rows == 0 && !sums) return ok();
  DeviceInfo dev;
  if ((rc = check_device(&dev)) != QKV_CTE_OK) return rc;
  LayerNormGradArgs a{};
  a.dy = dy;
  a.lddy = dy_row_stride;
  a.x = x;
  a.ldx = x_row_stride;
  a.weight = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  a.lddx = dx_row_stride;
  a.dweight = dweight;
  a.dbias = dbias;
  a.partial = sums ? static_cast<float*>(workspace) : nullptr;
  a.max_parts = kLayerNormMaxParts;
  a.rows = rows;
  a.cols = cols;
  const cudaError_t err = launch_layer_norm_backward(a, dtype, param_dtype, sums, static_cast<cudaStream_t>(stream), dev.sms);
  if (err != cudaSuccess) return fail(QKV_CTE_ERR_CUDA, "layer norm backward launch: %s", cudaGetErrorString(err));
  return ok();
}

}  // extern "C"

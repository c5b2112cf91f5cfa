// Argument checks of strided [batch, seq, heads, d] tensors, shared by the C-ABI front ends.
#pragma once

#include <climits>
#include <cstddef>
#include <cstdint>
#include <utility>

#include "api_common.h"

namespace qkvcte {

// Strides in elements; the d lanes are contiguous.
struct HeadsView {
  const void* p;
  int64_t sb, ss, sh;
  int64_t batch, seq, heads, d;
  size_t elem;
};

// Null, alignment to the element, strides; *bytes: from the first element to the last.
// `distinct` demands that no two elements share an address.
inline int check_heads(const HeadsView& t, bool distinct, const char* name, const char* who, size_t* bytes) {
  if (t.p == nullptr) return fail(QKV_CTE_ERR_INVALID, "%s: null %s", who, name);
  if (!aligned(t.p, t.elem))
    return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: %s is not aligned to its elements", who, name);
  struct Dim {
    int64_t stride, size;
  } dims[3] = {{t.sb, t.batch}, {t.ss, t.seq}, {t.sh, t.heads}};
  for (int i = 1; i < 3; ++i)  // by stride, ascending
    for (int j = i; j > 0 && dims[j].stride < dims[j - 1].stride; --j) std::swap(dims[j], dims[j - 1]);
  int64_t extent = t.d;
  for (const Dim& v : dims) {
    if (v.size <= 1) continue;
    if (v.stride < 0) return fail(QKV_CTE_ERR_INVALID, "%s: negative stride of %s", who, name);
    if (distinct && v.stride < extent)
      return fail(QKV_CTE_ERR_INVALID, "%s: the strides of %s make its elements overlap", who, name);
    if (v.stride > (INT64_MAX / 16 - extent) / (v.size - 1))
      return fail(QKV_CTE_ERR_UNSUPPORTED, "%s: size of %s overflows", who, name);
    extent += v.stride * (v.size - 1);
  }
  *bytes = static_cast<size_t>(extent) * t.elem;
  return QKV_CTE_OK;
}

// Whether two checked tensors of the same batch and seq share a byte. Two column ranges of
// one wide [batch * seq, ...] tensor lie side by side and do not.
inline bool heads_overlap(const HeadsView& x, size_t x_bytes, const HeadsView& y, size_t y_bytes) {
  if (!overlaps(x.p, x_bytes, y.p, y_bytes)) return false;
  const bool rows = (x.batch == 1 || (x.sb == x.seq * x.ss && y.sb == y.seq * y.ss)) &&
                    (x.heads == 1 || x.sh >= 0) && (y.heads == 1 || y.sh >= 0);
  const int64_t xr = ((x.heads > 1 ? (x.heads - 1) * x.sh : 0) + x.d) * static_cast<int64_t>(x.elem);
  const int64_t yr = ((y.heads > 1 ? (y.heads - 1) * y.sh : 0) + y.d) * static_cast<int64_t>(y.elem);
  const int64_t xs = x.ss * static_cast<int64_t>(x.elem), ys = y.ss * static_cast<int64_t>(y.elem);
  return !rows || xr > xs || yr > ys || strided_rows_overlap(x.p, xs, y.p, ys, x.batch * x.seq, xr, yr);
}

}  // namespace qkvcte

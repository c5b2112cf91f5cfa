// Helpers shared by the C-ABI front ends (defined in qkv_cte_api.cu): the thread's last
// error, device checks, pointer checks and operand tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "qkv_cte.h"

namespace qkvcte {

struct DeviceInfo {
  bool init = false;
  int major = 0, minor = 0, sms = 0;
};

// Record the message behind qkv_cte_last_error() and return `code`.
__attribute__((format(printf, 2, 3))) int fail(int code, const char* fmt, ...);
// Clear the message; QKV_CTE_OK.
int ok();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The current device, refused unless it is sm_103.
int check_device(DeviceInfo* dev);

// Whether [a, a + na) and [b, b + nb) share a byte (null or empty: no).
bool overlaps(const void* a, size_t na, const void* b, size_t nb);

// Whether two blocks of `rows` rows share a byte: rows of a_row (b_row, or the same) bytes,
// a_stride and b_stride bytes apart. Blocks of one stride whose rows lie side by side (two
// column ranges of one wide tensor) do not.
bool strided_rows_overlap(const void* a, int64_t a_stride, const void* b, int64_t b_stride, int64_t rows,
                          int64_t a_row, int64_t b_row = 0);

// 2D K-major uint8 operand [rows, cols], tiles of box_rows x 128 bytes, 128-byte swizzle.
int encode_operand(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows,
                   const char* what);
// The repacked weight scales of `g` (see launch_prep), one 128-byte K block per box.
struct GemmShape;
int encode_scales(CUtensorMap* m, void* base, const GemmShape& g);

// N tiles per band of the GEMM's tile order.
int band_tiles(const GemmShape& g);

}  // namespace qkvcte

// Kernel K1 (CTA-pair form) with the product's epilogue: bias, activation, gate and
// residual, outputs of a 16-bit type, in a translation unit of its own.
#include "qkv_cte.h"
#include "qkv_gemm_mxf8.cuh"

namespace qkvcte {

cudaError_t launch_gemm_linear(const GemmShape& g, const CUtensorMap& tmA, const CUtensorMap& tmW,
                               const CUtensorMap& tmSF, const GemmArgs& a, cudaStream_t s, int num_sms) {
  if (a.lin.dtype == QKV_CTE_DTYPE_FP32) return launch_gemm_linear_f32(g, tmA, tmW, tmSF, a, s, num_sms);
  const NormRopeArgs none{};
  switch (g.tile_n) {
    case 128: return launch_gemm_pair_t<128, kEpiLinear, false>(g, tmA, tmW, tmSF, a, none, s, num_sms);
    case 192: return launch_gemm_pair_t<192, kEpiLinear, false>(g, tmA, tmW, tmSF, a, none, s, num_sms);
    case 240: return launch_gemm_pair_t<240, kEpiLinear, false>(g, tmA, tmW, tmSF, a, none, s, num_sms);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qkvcte

// Kernel K1 (CTA-pair form) with the product's epilogue and fp32 outputs.
#include "qkv_gemm_mxf8.cuh"

namespace qkvcte {

cudaError_t launch_gemm_linear_f32(const GemmShape& g, const CUtensorMap& tmA, const CUtensorMap& tmW,
                                   const CUtensorMap& tmSF, const GemmArgs& a, cudaStream_t s, int num_sms) {
  const NormRopeArgs none{};
  switch (g.tile_n) {
    case 128: return launch_gemm_pair_t<128, kEpiLinearF32, false>(g, tmA, tmW, tmSF, a, none, s, num_sms);
    case 192: return launch_gemm_pair_t<192, kEpiLinearF32, false>(g, tmA, tmW, tmSF, a, none, s, num_sms);
    case 240: return launch_gemm_pair_t<240, kEpiLinearF32, false>(g, tmA, tmW, tmSF, a, none, s, num_sms);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qkvcte

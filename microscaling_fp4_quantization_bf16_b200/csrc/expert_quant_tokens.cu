// expert_quant_tokens.cu -- tokens quantized into expert order.
#include "expert_quant.cuh"

namespace fp4q {
cudaError_t launch_token_quant(int strat, int rot, const RowQuantArgs& a, cudaStream_t st)
{
    FP4Q_ROWS_ROTS(token_quant_kernel, 16, K_ABSMAX)
    FP4Q_ROWS_ROTS(token_quant_kernel, 16, K_PREVENT_ZERO)
    FP4Q_ROWS_ROTS(token_quant_kernel, 16, K_FOUR_OVER_SIX)
    FP4Q_ROWS_ROTS(token_quant_kernel, 16, K_BRUTE_FORCE)
    FP4Q_ROWS_ROTS(token_quant_kernel, 32, K_MX)
    FP4Q_ROWS_ROTS(token_quant_kernel, 32, K_MX_BRUTE)
    return cudaErrorInvalidValue;
}
}  // namespace fp4q

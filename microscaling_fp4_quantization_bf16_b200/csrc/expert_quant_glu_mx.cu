// expert_quant_glu_mx.cu -- gated activation quantized to MXFP4.
#include "expert_quant.cuh"

namespace fp4q {
cudaError_t launch_glu_quant_mx(int strat, int rot, const RowQuantArgs& a, cudaStream_t st)
{
    FP4Q_GLU_ROTS(32, K_MX)
    FP4Q_GLU_ROTS(32, K_MX_BRUTE)
    return cudaErrorInvalidValue;
}
}  // namespace fp4q

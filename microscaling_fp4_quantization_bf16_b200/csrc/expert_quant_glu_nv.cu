// expert_quant_glu_nv.cu -- gated activation quantized to NVFP4, and its abs-max.
#include "expert_quant.cuh"

namespace fp4q {

namespace {

template <int ROT, int ACT>
__global__ void __launch_bounds__(QTHREADS) glu_amax_kernel(RowQuantArgs a, uint32_t ntiles)
{
    pdl_begin();
    const int lane = threadIdx.x & 31;
    __shared__ uint4 in[QTHREADS / 32][2][2][32 * 4];
    unsigned m = 0;
    glu_tiles<ACT>(a, ntiles, lane, in[threadIdx.x / 32], [&](float (&y)[SEG], const Place&, int32_t) {
        rotate_seg<ROT>(y, lane);
        m = max(m, seg_amax(y));
    });
    put_amax(a, m);
}

template <int ROT>
cudaError_t glu_amax_act(const RowQuantArgs& a, int* parts, cudaStream_t st)
{
    return a.act == FP4Q_ACT_SILU
               ? launch_rows<glu_amax_kernel<ROT, FP4Q_ACT_SILU>>(a, st, FP4Q_AMAX_WORK, parts)
               : launch_rows<glu_amax_kernel<ROT, FP4Q_ACT_GELU_TANH>>(a, st, FP4Q_AMAX_WORK, parts);
}

}  // namespace

cudaError_t launch_glu_amax(int rot, const RowQuantArgs& a, int* parts, cudaStream_t st)
{
    switch (rot) {
    case 0: return glu_amax_act<0>(a, parts, st);
    case 16: return glu_amax_act<16>(a, parts, st);
    case 32: return glu_amax_act<32>(a, parts, st);
    case 64: return glu_amax_act<64>(a, parts, st);
    case 128: return glu_amax_act<128>(a, parts, st);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_glu_quant_nv(int strat, int rot, const RowQuantArgs& a, cudaStream_t st)
{
    FP4Q_GLU_ROTS(16, K_ABSMAX)
    FP4Q_GLU_ROTS(16, K_PREVENT_ZERO)
    FP4Q_GLU_ROTS(16, K_FOUR_OVER_SIX)
    FP4Q_GLU_ROTS(16, K_BRUTE_FORCE)
    return cudaErrorInvalidValue;
}
}  // namespace fp4q

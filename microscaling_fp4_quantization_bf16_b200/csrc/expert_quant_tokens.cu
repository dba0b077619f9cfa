// expert_quant_tokens.cu -- tokens quantized into expert order.
#include "expert_quant.cuh"

namespace fp4q {

namespace {

template <int ROT>
__global__ void __launch_bounds__(QTHREADS) token_amax_kernel(RowQuantArgs a, int64_t ntiles)
{
    pdl_begin();
    const int lane = threadIdx.x & 31;
    unsigned m = 0;
    int64_t s = (int64_t)blockIdx.x * QTHREADS + threadIdx.x;
    for (int64_t t = blockIdx.x; t < ntiles; t += gridDim.x, s += (int64_t)gridDim.x * QTHREADS) {
        if (s - lane >= a.nseg)  // warp-uniform
            break;
        float y[SEG];
        load_seg_bf16(a.x, a.nseg * SEG, s, y);  // past the end reads zeros
        rotate_seg<ROT>(y, lane);
        m = max(m, seg_amax(y));
    }
    put_amax(a, m);
}

}  // namespace

cudaError_t launch_token_amax(int rot, const RowQuantArgs& a, int* parts, cudaStream_t st)
{
    switch (rot) {
    case 0: return launch_rows<token_amax_kernel<0>>(a, st, FP4Q_AMAX_WORK, parts);
    case 16: return launch_rows<token_amax_kernel<16>>(a, st, FP4Q_AMAX_WORK, parts);
    case 32: return launch_rows<token_amax_kernel<32>>(a, st, FP4Q_AMAX_WORK, parts);
    case 64: return launch_rows<token_amax_kernel<64>>(a, st, FP4Q_AMAX_WORK, parts);
    case 128: return launch_rows<token_amax_kernel<128>>(a, st, FP4Q_AMAX_WORK, parts);
    default: return cudaErrorInvalidValue;
    }
}

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

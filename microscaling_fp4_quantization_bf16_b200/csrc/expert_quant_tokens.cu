// expert_quant_tokens.cu -- tokens quantized into expert order.
#include "expert_quant.cuh"

namespace fp4q {

namespace {

// Without a rotation the maximum is taken on the packed bf16 magnitudes, 16
// bytes a lane and load, eight of them in flight.
template <int ROT>
__global__ void __launch_bounds__(QTHREADS) token_amax_kernel(RowQuantArgs a, uint32_t ntiles)
{
    pdl_begin();
    const int lane = threadIdx.x & 31;
    unsigned m = 0;
    if constexpr (ROT == 0) {
        constexpr int FLIGHT = 8;
        const uint4* x4 = reinterpret_cast<const uint4*>(a.x);
        const int64_t n4 = (int64_t)a.nseg * 4, step = (int64_t)gridDim.x * QTHREADS * FLIGHT;
        // a warp's loads cover 4 KB together
        for (int64_t i = ((int64_t)blockIdx.x * QTHREADS + threadIdx.x - lane) * FLIGHT + lane; i < n4;
             i += step) {
            uint4 v[FLIGHT];
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k)
                v[k] = i + 32 * k < n4 ? ldg_stream(x4 + i + 32 * k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < FLIGHT; ++k) {
                m = __vmaxu2(m, __vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu));
                m = __vmaxu2(m, __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu));
            }
        }
        m = max(m & 0xFFFFu, m >> 16) << 16;
    } else {
        const uint32_t step = gridDim.x * QTHREADS;
        uint32_t s = blockIdx.x * QTHREADS + threadIdx.x;
        for (uint32_t t = blockIdx.x; t < ntiles; t += gridDim.x, s += step) {
            if (s - lane >= a.nseg)  // warp-uniform
                break;
            float y[SEG];
            load_seg_bf16(a.x, (int64_t)a.nseg * SEG, s, y);  // past the end reads zeros
            rotate_seg<ROT>(y, lane);
            m = max(m, seg_amax(y));
        }
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

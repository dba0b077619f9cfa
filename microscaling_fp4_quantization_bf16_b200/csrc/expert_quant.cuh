// expert_quant.cuh -- rows quantized into the block-scaled MMA layout at the
// rows that the expert order gives them.
//
// Arithmetic: process_segment of quant_kernel.cuh, one thread to a 32-element
// segment, so codes, scales and values are bit for bit those of the plain
// quantizer. It writes into a small shared-memory buffer of the warp instead
// of global memory (its pointers are generic); from there a token's segment goes to
// each of its k rows, so a token is read and quantized once however many
// experts take it, and the 64-byte (bf16) or 128-byte (fp32) pieces of the
// values leave as 512 contiguous bytes a warp.
#pragma once

#include "experts.h"
#include "quant_kernel.cuh"

namespace fp4q {

// One warp's staging buffer: 32 segments' codes, scale bytes and values.
template <int B>
struct WarpStage {
    uint4 codes[32];
    uint8_t scales[32 * (SEG / B)];
    __align__(16) uint8_t dq[32 * SEG * sizeof(float)];
};

// The destination rows of one segment's choice j; -1 where there is none.
__device__ __forceinline__ int32_t row_of(const RowQuantArgs& a, int64_t i, int j)
{
    int32_t r = a.slots == nullptr ? (int32_t)i : a.slots[i * a.k + j];
    return r < a.rows ? r : -1;
}

// Copies the staged segments of a warp to their rows. i, p: token (or taken
// row) and segment within it of this lane; live: the lane has a segment. All lanes take part.
template <int B>
__device__ __forceinline__ void store_rows(const RowQuantArgs& a, const WarpStage<B>& st, int lane,
                                           int64_t i, uint32_t p, bool live)
{
    constexpr int NB = SEG / B;      // blocks of a segment
    constexpr int QUAD = 4 / NB;     // segments of a 4-block group
    const uint4 q = st.codes[lane];
    // Segments per row a multiple of QUAD: the groups of 4 blocks lie inside
    // the warp, and the first lane of each writes its 4 bytes at once.
    const bool whole = a.spr % QUAD == 0;
    uint32_t quad = 0;
    if (whole && lane % QUAD == 0)
        quad = *reinterpret_cast<const uint32_t*>(st.scales + lane * NB);
    for (int j = 0; j < a.k; ++j) {
        const int32_t r = live ? row_of(a, i, j) : -1;
        if (r >= 0) {
            *reinterpret_cast<uint4*>(a.codes + ((int64_t)r * a.spr + p) * (SEG / 2)) = q;
            const uint32_t kb = p * NB;
            uint8_t* dst = a.scales + ((int64_t)(r >> 7) * a.atoms_k + (kb >> 2)) * 512 +
                           16 * (r & 31) + 4 * ((r >> 5) & 3);
            if (whole) {
                if (lane % QUAD == 0)
                    *reinterpret_cast<uint32_t*>(dst) = quad;
            } else {
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    dst[(kb & 3) + b] = st.scales[lane * NB + b];
                if (p == a.spr - 1)  // padding blocks of the row's last group
                    for (uint32_t b = (kb & 3) + NB; b < 4; ++b)
                        dst[b] = 0;
            }
        }
        if (a.dq_kind == 0)  // uniform
            continue;
        const int bytes = a.dq_kind == 1 ? 4 * SEG : 2 * SEG;  // of a segment's values
        const int per = bytes / 16;
        for (int c = lane; c < 32 * per; c += 32) {
            const int sl = c / per;
            const int32_t rs = __shfl_sync(0xFFFFFFFFu, r, sl);
            const uint32_t ps = __shfl_sync(0xFFFFFFFFu, p, sl);
            if (rs >= 0)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.dq) +
                                          ((int64_t)rs * a.spr + ps) * bytes + 16 * (c % per)) =
                    *reinterpret_cast<const uint4*>(st.dq + 16 * c);
        }
    }
}

// The staging buffer as the output of process_segment.
template <int B>
__device__ __forceinline__ QuantArgs stage_args(const RowQuantArgs& a, WarpStage<B>& st)
{
    QuantArgs q;
    q.x = nullptr;
    q.n = 0;
    q.amax = a.amax;
    q.sg_out = a.sg_out;
    q.codes = reinterpret_cast<uint8_t*>(st.codes);
    q.scales = st.scales;
    q.mse = nullptr;
    q.dq = st.dq;
    q.dq_kind = a.dq_kind;
    q.keep = a.keep;
    q.mma_spr = 0;
    q.mma_atoms_k = 0;
    return q;
}

// The tensor abs-max that build_scale_tables reads, from the maxima of the
// abs-max pass's CTAs (every CTA takes their maximum itself: no launch
// in between, no value to clear beforehand). Ends with a CTA barrier.
__device__ __forceinline__ void join_amax(const RowQuantArgs& a, float& joined, QuantArgs& q)
{
    if (a.amax_parts == 0)  // uniform
        return;
    __shared__ unsigned top[QTHREADS / 32];
    unsigned m = 0;
    for (int i = threadIdx.x; i < a.amax_parts; i += QTHREADS)
        m = max(m, __float_as_uint(a.amax[i]));
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (threadIdx.x % 32 == 0)
        top[threadIdx.x / 32] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < QTHREADS / 32; ++w)
            m = max(m, top[w]);
        joined = __uint_as_float(m);
    }
    __syncthreads();
    q.amax = &joined;
}

// Writes the CTA's maximum of m (bits of non-negative floats).
__device__ __forceinline__ void put_amax(const RowQuantArgs& a, unsigned m)
{
    __shared__ unsigned top[QTHREADS / 32];
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (threadIdx.x % 32 == 0)
        top[threadIdx.x / 32] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < QTHREADS / 32; ++w)
            m = max(m, top[w]);
        a.amax_out[blockIdx.x] = __uint_as_float(m);
    }
}

__device__ __forceinline__ unsigned seg_amax(const float (&y)[SEG])
{
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < SEG; ++k)
        m = fmaxf(m, fabsf(y[k]));
    return __float_as_uint(m);
}

template <int STRAT>
struct RowMinBlocks {
    static constexpr int value = STRAT == K_BRUTE_FORCE || STRAT == K_MX_BRUTE ? 1 : 5;
};

// Tokens: segment s of x is segment s % spr of token s / spr. Persistent CTAs;
// the next tile's loads are in flight during this tile's arithmetic.
template <int B, int ROT, int STRAT>
__global__ void __launch_bounds__(QTHREADS, RowMinBlocks<STRAT>::value)
    token_quant_kernel(RowQuantArgs a, int64_t ntiles)
{
    pdl_begin();
    __shared__ ScaleTables<STRAT> tab;
    __shared__ WarpStage<B> stage[QTHREADS / 32];
    const int lane = threadIdx.x & 31;
    WarpStage<B>& st = stage[threadIdx.x / 32];
    QuantArgs qa = stage_args<B>(a, st);
    __shared__ float joined;
    const uint4* x4 = reinterpret_cast<const uint4*>(a.x);
    auto fetch = [&](int64_t s, uint4 (&raw)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            raw[k] = s < a.nseg ? ldg_stream(x4 + 4 * s + k) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 raw[4];
    int64_t s = (int64_t)blockIdx.x * QTHREADS + threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * QTHREADS;
    fetch(s, raw);
    join_amax(a, joined, qa);
    build_scale_tables<STRAT>(tab, qa);
    for (int64_t t = blockIdx.x; t < ntiles; t += gridDim.x, s += step) {
        float y[SEG];
        unpack_seg<!is_mx_strat(STRAT)>(raw, y);
        if (t + gridDim.x < ntiles)
            fetch(s + step, raw);
        if (s - lane < a.nseg) {  // warp-uniform
            rotate_seg<ROT, !foldable<ROT, STRAT>()>(y, lane);
            process_segment<B, STRAT, ROT>(y, lane, SEG, qa, tab);
            __syncwarp();
            const uint32_t i = (uint32_t)s / a.spr;
            store_rows<B>(a, st, lane, i, (uint32_t)s - i * a.spr, s < a.nseg);
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------- gated activation

// h = bf16(fp32(g u sigmoid(z))) from its real value: 64 bits, one rounding to
// fp32, one to bf16. Only pairs whose rounding the fp32 path cannot decide come here.
static __device__ __noinline__ uint32_t glu_pair_exact(uint32_t g2, uint32_t u2, int act)
{
    uint32_t out = 0;
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        const double g = (double)__uint_as_float(k ? g2 & 0xFFFF0000u : g2 << 16);
        const double u = (double)__uint_as_float(k ? u2 & 0xFFFF0000u : u2 << 16);
        const double z = act == FP4Q_ACT_GELU_TANH
                             ? 1.5957691216057307612 * (g + 0.044715 * g * g * g)
                             : g;
        const float h = (float)(g * u / (1.0 + exp(-z)));
        out |= (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(h)) << (16 * k);
    }
    return out;
}

// Two values of h as packed bf16, from packed bf16 gates and values.
//
// v = (g u) / (1 + 2^(-z log2 e)) in fp32 with the hardware's 2^x and 1/x is
// within E |v| of the real value: 2^x is off by 2^-22.5 and its argument
// by 2^-23.4 |z| (products and constant), which count in full only where z < 0;
// the sum, the reciprocal and two products add 2^-22 at most; gelu's z itself is off by 2^-22 |z|.
// E = 2^-20 + 2^-21 max(-z, 0) covers all of it. The ends v (1 -+ E) of that
// bracket round to the same bf16 in all but about one pair in a thousand; those, and
// whatever leaves the range in which relative errors hold, are formed in 64 bits.
__device__ __forceinline__ uint32_t glu_pair(uint32_t g2, uint32_t u2, bool gelu, int act)
{
    uint32_t lo[2];
    bool ok = true;
    float b[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float g = k ? bf_hi(g2) : bf_lo(g2);
        const float u = k ? bf_hi(u2) : bf_lo(u2);
        float z = g;
        if (gelu)
            z = (1.5957691216f * g) * __fmaf_rn(0.044715f * g, g, 1.0f);
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950409f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
        const float v = (g * u) * r;
        const float err = __fmaf_rn(fmaxf(-z, 0.0f), 0x1p-21f, 0x1p-20f);
        b[0][k] = __fmaf_rn(v, -err, v);
        b[1][k] = __fmaf_rn(v, err, v);
        // z > -60 keeps 2^x and its reciprocal in range, |v| > 2^-100 the products
        // (g u and v differ by a factor above 2^-88); a zero factor is exact
        ok = ok && z > -60.0f && (fabsf(v) > 0x1p-100f || g == 0.0f || u == 0.0f);
    }
    lo[0] = pack_bf16x2(b[0][0], b[0][1]);
    lo[1] = pack_bf16x2(b[1][0], b[1][1]);
    if (ok && lo[0] == lo[1])
        return lo[0];
    return glu_pair_exact(g2, u2, act);
}

// The 32 values of one segment of h, widened; row < 0 gives zeros.
__device__ __forceinline__ void load_glu(const RowQuantArgs& a, int64_t row, uint32_t p, float (&y)[SEG])
{
    if (row < 0) {
#pragma unroll
        for (int i = 0; i < SEG; ++i)
            y[i] = 0.0f;
        return;
    }
    const uint4* g4 = reinterpret_cast<const uint4*>(a.x) + ((int64_t)row * 2 * a.spr + p) * 4;
    const uint4* u4 = g4 + (int64_t)a.spr * 4;
    uint4 g[4], u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        g[k] = ldg_stream(g4 + k);
        u[k] = ldg_stream(u4 + k);
    }
    const bool gelu = a.act == FP4Q_ACT_GELU_TANH;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t gw[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
        const uint32_t uw[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const uint32_t h = glu_pair(gw[w], uw[w], gelu, a.act);
            y[8 * k + 2 * w] = bf_lo(h);
            y[8 * k + 2 * w + 1] = bf_hi(h);
        }
    }
}

template <int B, int ROT, int STRAT>
__global__ void __launch_bounds__(QTHREADS, RowMinBlocks<STRAT>::value)
    glu_quant_kernel(RowQuantArgs a, int64_t ntiles)
{
    pdl_begin();
    __shared__ ScaleTables<STRAT> tab;
    __shared__ WarpStage<B> stage[QTHREADS / 32];
    const int lane = threadIdx.x & 31;
    WarpStage<B>& st = stage[threadIdx.x / 32];
    QuantArgs qa = stage_args<B>(a, st);
    __shared__ float joined;
    join_amax(a, joined, qa);
    build_scale_tables<STRAT>(tab, qa);
    int64_t s = (int64_t)blockIdx.x * QTHREADS + threadIdx.x;
    for (int64_t t = blockIdx.x; t < ntiles; t += gridDim.x, s += (int64_t)gridDim.x * QTHREADS) {
        if (s - lane >= a.nseg)  // warp-uniform
            break;
        const bool live = s < a.nseg;
        const uint32_t i = (uint32_t)s / a.spr;
        const uint32_t p = (uint32_t)s - i * a.spr;
        float y[SEG];
        load_glu(a, live ? row_of(a, i, 0) : -1, p, y);
        rotate_seg<ROT, !foldable<ROT, STRAT>()>(y, lane);
        process_segment<B, STRAT, ROT>(y, lane, SEG, qa, tab);
        __syncwarp();
        store_rows<B>(a, st, lane, i, p, live);
        __syncwarp();
    }
}

// Launch of a row quantize kernel over the resident CTAs, at most `most`.
template <class K>
cudaError_t launch_rows(K kernel, const RowQuantArgs& a, cudaStream_t st, int64_t most = 0x7FFFFFFF,
                        int* ctas = nullptr)
{
    const int64_t nblk = (a.nseg + QTHREADS - 1) / QTHREADS;
    const int64_t res = resident_ctas(kernel);
    if (res < 0)
        return cudaErrorUnknown;
    int64_t grid = nblk < res ? nblk : res;
    grid = grid < most ? grid : most;
    if (ctas != nullptr)
        *ctas = (int)grid;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(QTHREADS), 0, st, a, nblk);
}

#define FP4Q_ROWS_CASE(KERNEL_, B_, S_, R_) \
    if (strat == S_ && rot == R_)           \
        return launch_rows(KERNEL_<B_, R_, S_>, a, st);
#define FP4Q_ROWS_ROTS(KERNEL_, B_, S_)  \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 0)   \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 16)  \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 32)  \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 64)  \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 128)

}  // namespace fp4q

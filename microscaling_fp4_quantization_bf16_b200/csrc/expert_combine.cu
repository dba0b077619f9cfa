// expert_combine.cu -- expert outputs back to tokens, and the gradients that
// run the other way: the weighted sum and its gradient, and the gradient of
// the gated activation.
//
// All are bound by memory: every value is read or written once, in 16-byte
// pieces of 8 values a thread, neighbouring threads on neighbouring pieces, so
// a warp's access covers 512 contiguous bytes. Sums run in a fixed order, in fp32, the router's
// gradient in 64 bits.
// A blockwise rotation (gradients are linear in it) runs on this layout: three
// butterfly stages inside a thread's 8 values, the others between lanes.
#include "experts.h"
#include "fp4q_device.cuh"

namespace fp4q {

namespace {

// Small CTAs: they retire and refill one by one (combine of 8192 tokens x 4096,
// eight experts each: 102 us with 128 threads, 104 with 256, 168 with 512).
constexpr int CTHREADS = 128;

// 8 consecutive values of a bf16 or fp32 array, element index i (multiple of 8)
template <bool F32>
struct Piece {
    uint4 w[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Piece<F32> load8(const void* p, int64_t i)
{
    Piece<F32> r;
    if constexpr (F32) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
        r.w[0] = ldg_stream(q);
        r.w[1] = ldg_stream(q + 1);
    } else {
        r.w[0] = ldg_stream(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ void widen8(const Piece<F32>& r, float (&v)[8])
{
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
    if constexpr (F32) {
        const uint32_t h[4] = {r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(w[i]);
            v[4 + i] = __uint_as_float(h[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf_lo(w[i]);
            v[2 * i + 1] = bf_hi(w[i]);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8])
{
    if constexpr (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 w;
        w.x = pack_bf16x2(v[0], v[1]);
        w.y = pack_bf16x2(v[2], v[3]);
        w.z = pack_bf16x2(v[4], v[5]);
        w.w = pack_bf16x2(v[6], v[7]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = w;
    }
}

// Normalised Walsh-Hadamard transform of ROT-wide chunks held 8 values a
// lane; every lane of the warp takes part, a chunk's ROT / 8 lanes are neighbours.
template <int ROT>
__device__ __forceinline__ void rotate8(float (&v)[8], int lane)
{
    if constexpr (ROT > 0) {
#pragma unroll
        for (int h = 1; h < 8; h *= 2)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((i & h) == 0) {
                    const float a = v[i], b = v[i + h];
                    v[i] = __fadd_rn(a, b);
                    v[i + h] = __fsub_rn(a, b);
                }
#pragma unroll
        for (int h = 1; h < ROT / 8; h *= 2) {
            const float sign = (lane & h) ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __fmaf_rn(sign, v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], h));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __fmul_rn(v[i], HadK<ROT>::k);
    }
}

// One thread: 8 columns of one token. The rows of up to GROUP choices are in
// flight together (8 of them cost the warps that hide more: 121 us against 104
// for 8192 tokens x 4096, eight experts each; 2 are too few, 111 us).
template <bool Y32, bool O32, int ROT>
__global__ void __launch_bounds__(CTHREADS) combine_kernel(CombineArgs a)
{
    constexpr int GROUP = 4;
    pdl_begin();
    const int64_t vpr = a.cols / 8;
    const int64_t i = (int64_t)blockIdx.x * CTHREADS + threadIdx.x;
    const bool live = i < a.tokens * vpr;
    const int64_t t = live ? i / vpr : 0;
    const int64_t c = live ? (i - t * vpr) * 8 : 0;
    const int32_t* slot = a.slots + t * a.k;
    float sum[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += GROUP) {
        int32_t r[GROUP];
        Piece<Y32> p[GROUP];
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
            r[j] = live && j0 + j < a.k ? slot[j0 + j] : -1;
            if (r[j] >= a.rows)
                r[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < GROUP; ++j)
            if (r[j] >= 0)
                p[j] = load8<Y32>(a.y, (int64_t)r[j] * a.cols + c);
#pragma unroll
        for (int j = 0; j < GROUP; ++j)
            if (r[j] >= 0) {
                const float w = a.weights != nullptr ? a.weights[t * a.k + j0 + j] : 1.0f;
                float v[8];
                widen8<Y32>(p[j], v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] = __fmaf_rn(w, v[e], sum[e]);
            }
    }
    rotate8<ROT>(sum, threadIdx.x & 31);
    if (live)
        store8<O32>(a.out, t * a.cols + c, sum);
}

// One block: one token. Each thread walks the token's columns 8 at a time:
// one read of g, one of each choice's row, one write of each choice's
// gradient; the products with y stay in one 64-bit accumulator per choice (a
// router's gradient is one number out of thousands of terms that may cancel), taken in 64 bits too: bf16
// has fp32's exponents, so a product of two may be out of its range (4000 tokens x 4096 to four experts:
// 48.7 us back to back; with the products of two bf16 numbers in fp32 46.9). Four choices at a time: more
// of them in flight cost registers and thereby warps (cold, with fp32 products: 52 us; 8 choices 67,
// two pieces of columns as well 61, both 104); of bf16 arrays 7 CTAs an SM (without the bound 49.2).
template <bool G32, bool Y32>
__global__ void __launch_bounds__(CTHREADS, G32 || Y32 ? 0 : 7) combine_bwd_kernel(CombineBwdArgs a)
{
    constexpr int GROUP = 4;
    pdl_begin();
    __shared__ double part[GROUP][CTHREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    const int64_t t = blockIdx.x;
    for (int j0 = 0; j0 < a.k; j0 += GROUP) {
        int32_t r[GROUP];
        float w[GROUP];
        double acc[GROUP];
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
            const bool in = j0 + j < a.k;
            r[j] = in ? a.slots[t * a.k + j0 + j] : -1;
            w[j] = in && a.weights != nullptr ? a.weights[t * a.k + j0 + j] : 1.0f;
            if (r[j] >= a.rows)
                r[j] = -1;
            acc[j] = 0.0;
        }
        for (int64_t c = threadIdx.x * 8; c < a.cols; c += blockDim.x * 8) {
            Piece<Y32> p[GROUP];
            const Piece<G32> gp = load8<G32>(a.g, t * a.cols + c);
            if (a.dw != nullptr) {
#pragma unroll
                for (int j = 0; j < GROUP; ++j)
                    if (r[j] >= 0)
                        p[j] = load8<Y32>(a.y, (int64_t)r[j] * a.cols + c);
            }
            float g[8];
            widen8<G32>(gp, g);
#pragma unroll
            for (int j = 0; j < GROUP; ++j)
                if (r[j] >= 0) {
                    float v[8];
                    if (a.dw != nullptr) {
                        widen8<Y32>(p[j], v);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            acc[j] = __fma_rn((double)g[e], (double)v[e], acc[j]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = __fmul_rn(w[j], g[e]);
                    store8<Y32>(a.dy, (int64_t)r[j] * a.cols + c, v);
                }
        }
        if (a.dw != nullptr) {
#pragma unroll
            for (int j = 0; j < GROUP; ++j) {
#pragma unroll
                for (int d = 16; d > 0; d /= 2)
                    acc[j] = __dadd_rn(acc[j], __shfl_xor_sync(0xFFFFFFFFu, acc[j], d));
                if (lane == 0)
                    part[j][warp] = acc[j];
            }
            __syncthreads();
            if (threadIdx.x < GROUP && j0 + (int)threadIdx.x < a.k) {
                double s = 0.0;
                for (int x = 0; x < warps; ++x)
                    s = __dadd_rn(s, part[threadIdx.x][x]);
                a.dw[t * a.k + j0 + threadIdx.x] = (float)s;
            }
            if (j0 + GROUP < a.k)
                __syncthreads();
        }
    }
}

// sigmoid(z) in fp32: a few units in the last place; 0 where it is below 2^-126 (z below -87.3).
__device__ __forceinline__ float sigmoid(float z)
{
    return __fdividef(1.0f, __fadd_rn(1.0f, __expf(-z)));
}

// The gate's gradients of one thread again, d[e] in and out, where one of them is not finite: g^2 is
// held finite (beyond 2^50 s is 0 or 1, and z', infinite from 2^64 on, meets the zero s (1 - s)),
// and where d u overflows in front of a small a'(g), u a'(g) is taken first (u is above 1 there).
// A call, hardly ever made: with it and the check before it 45.5 -> 46.0 us (5821 x 4096, gelu,
// H16); inlined, its registers make that 50.
__device__ __noinline__ void far_gates(const uint16_t* g, const uint16_t* u, bool gelu, float* d)
{
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
        const float ge = bf_lo(g[e]), ue = bf_lo(u[e]);
        float z = ge, dz = 1.0f;
        if (gelu) {
            constexpr float C = 1.5957691216057308f;
            const float g2 = fminf(ge * ge, 0x1p100f);
            z = C * ge * __fmaf_rn(0.044715f, g2, 1.0f);
            dz = C * __fmaf_rn(3.0f * 0.044715f, g2, 1.0f);
        }
        const float s = sigmoid(z);
        const float da = __fmaf_rn(ge * s * (1.0f - s), dz, s);
        const float du = d[e] * ue;
        d[e] = fabsf(du) <= FLT_MAX ? du * da : d[e] * (ue * da);
    }
}

template <int ROT>
__global__ void __launch_bounds__(CTHREADS) glu_bwd_kernel(GluBwdArgs a)
{
    pdl_begin();
    const int64_t vpr = a.cols / 8;
    const int64_t i = (int64_t)blockIdx.x * CTHREADS + threadIdx.x;
    bool live = i < a.n * vpr;
    const int64_t t = live ? i / vpr : 0;
    const int64_t c = live ? (i - t * vpr) * 8 : 0;
    int64_t r = t;
    if (live && a.slots != nullptr) {
        r = a.slots[t];
        live = r >= 0 && r < a.rows;
    }
    float g[8] = {}, u[8] = {}, d[8] = {};
    if (live) {
        const Piece<false> pd = load8<false>(a.dh, r * a.cols + c);
        const Piece<false> pg = load8<false>(a.gu, r * 2 * a.cols + c);
        const Piece<false> pu = load8<false>(a.gu, r * 2 * a.cols + a.cols + c);
        widen8<false>(pd, d);
        widen8<false>(pg, g);
        widen8<false>(pu, u);
    }
    rotate8<ROT>(d, threadIdx.x & 31);
    if (!live)
        return;
    const bool gelu = a.act == FP4Q_ACT_GELU_TANH;
    float dg[8], du[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float z = g[e], dz = 1.0f;
        if (gelu) {
            constexpr float C = 1.5957691216057308f;  // 2 sqrt(2 / pi)
            const float g2 = g[e] * g[e];
            z = C * g[e] * __fmaf_rn(0.044715f, g2, 1.0f);
            dz = C * __fmaf_rn(3.0f * 0.044715f, g2, 1.0f);
        }
        const float s = sigmoid(z);
        const float as = g[e] * s;                     // a(g)
        const float da = __fmaf_rn(as * (1.0f - s), dz, s);
        du[e] = d[e] * as;
        dg[e] = d[e] * u[e] * da;
    }
    // one sum shows an infinity or NaN among them (or overflows itself)
    float s0, s1;
    upk2(add2(add2(pk2(dg[0], dg[1]), pk2(dg[2], dg[3])), add2(pk2(dg[4], dg[5]), pk2(dg[6], dg[7]))), s0, s1);
    if (!(fabsf(s0 + s1) <= FLT_MAX)) {
        const uint16_t* gate = a.gu + r * 2 * a.cols + c;
        float again[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            again[e] = d[e];
        far_gates(gate, gate + a.cols, gelu, again);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            dg[e] = again[e];
    }
    store8<false>(a.dgu, r * 2 * a.cols + c, dg);
    store8<false>(a.dgu, r * 2 * a.cols + a.cols + c, du);
}

cudaError_t grid_of(int64_t threads, unsigned* grid)
{
    const int64_t g = (threads + CTHREADS - 1) / CTHREADS;
    if (g <= 0 || g > 0x7FFFFFFF)
        return cudaErrorInvalidValue;
    *grid = (unsigned)g;
    return cudaSuccess;
}

template <bool Y32, bool O32>
cudaError_t combine_rot(int rot, const CombineArgs& a, unsigned grid, cudaStream_t st)
{
    switch (rot) {
    case 0: return launch_pdl(combine_kernel<Y32, O32, 0>, dim3(grid), dim3(CTHREADS), 0, st, a);
    case 16: return launch_pdl(combine_kernel<Y32, O32, 16>, dim3(grid), dim3(CTHREADS), 0, st, a);
    case 32: return launch_pdl(combine_kernel<Y32, O32, 32>, dim3(grid), dim3(CTHREADS), 0, st, a);
    case 64: return launch_pdl(combine_kernel<Y32, O32, 64>, dim3(grid), dim3(CTHREADS), 0, st, a);
    case 128: return launch_pdl(combine_kernel<Y32, O32, 128>, dim3(grid), dim3(CTHREADS), 0, st, a);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_combine(bool y32, bool out32, int rot, const CombineArgs& a, cudaStream_t st)
{
    unsigned grid = 0;
    if (cudaError_t e = grid_of(a.tokens * (a.cols / 8), &grid))
        return e;
    if (y32)
        return out32 ? combine_rot<true, true>(rot, a, grid, st)
                     : combine_rot<true, false>(rot, a, grid, st);
    return out32 ? combine_rot<false, true>(rot, a, grid, st)
                 : combine_rot<false, false>(rot, a, grid, st);
}

cudaError_t launch_combine_bwd(bool g32, bool y32, const CombineBwdArgs& a, cudaStream_t st)
{
    // a warp per 256 columns, at most CTHREADS threads
    const int64_t warps = (a.cols + 255) / 256;
    const int threads = 32 * (int)(warps < CTHREADS / 32 ? warps : CTHREADS / 32);
    const unsigned grid = (unsigned)a.tokens;  // below 2^31
    if (g32)
        return y32 ? launch_pdl(combine_bwd_kernel<true, true>, dim3(grid), dim3(threads), 0, st, a)
                   : launch_pdl(combine_bwd_kernel<true, false>, dim3(grid), dim3(threads), 0, st, a);
    return y32 ? launch_pdl(combine_bwd_kernel<false, true>, dim3(grid), dim3(threads), 0, st, a)
               : launch_pdl(combine_bwd_kernel<false, false>, dim3(grid), dim3(threads), 0, st, a);
}

cudaError_t launch_glu_bwd(int rot, const GluBwdArgs& a, cudaStream_t st)
{
    unsigned grid = 0;
    if (cudaError_t e = grid_of(a.n * (a.cols / 8), &grid))
        return e;
    switch (rot) {
    case 0: return launch_pdl(glu_bwd_kernel<0>, dim3(grid), dim3(CTHREADS), 0, st, a);
    case 16: return launch_pdl(glu_bwd_kernel<16>, dim3(grid), dim3(CTHREADS), 0, st, a);
    case 32: return launch_pdl(glu_bwd_kernel<32>, dim3(grid), dim3(CTHREADS), 0, st, a);
    case 64: return launch_pdl(glu_bwd_kernel<64>, dim3(grid), dim3(CTHREADS), 0, st, a);
    case 128: return launch_pdl(glu_bwd_kernel<128>, dim3(grid), dim3(CTHREADS), 0, st, a);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace fp4q

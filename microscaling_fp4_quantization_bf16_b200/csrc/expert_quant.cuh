// expert_quant.cuh -- rows quantized into the block-scaled MMA layout at the
// rows that the expert order gives them.
//
// Arithmetic: process_segment of quant_kernel.cuh, one thread to a 32-element
// segment, so codes, scales and values are bit for bit those of the plain
// quantizer under the same s_g. That is the same number for a given abs-max; without one it may be a
// unit in the last place apart (see row_scale_tables). A token is read and quantized once however
// many experts take it.
//
// Memory: each warp brings its next 32 segments (2 KB of bf16, twice that for
// gate and value) into shared memory with 16-byte asynchronous copies while it
// works on the current ones, 512 contiguous bytes a copy instruction (chunk c of
// segment s at slot c ^ (s / 2 % 4) of its four, so that reading a segment a
// lane is free of bank conflicts too). No register holds a byte in flight.
// process_segment leaves its codes and scale bytes in registers (its output
// pointers are a lane's own variables); from there a segment goes to each of its
// token's rows. Dequantized values, where they are wanted, are formed by the
// lane that stores them, from codes that pass through shared memory, again 512
// contiguous bytes an instruction. (One lane to a segment for loads and stores, 64
// bytes apart: 215 against 205 us for the activation of 8192 x 14336, 196
// against 188 for 16384 x 8192 tokens to two experts each.)
//
// Bound by: with values written, tokens by memory (16384 x 8192 to two experts
// each, 4-over-6: 936 MB in 184 us, 5.1 TB/s, seven tenths writes); without,
// by instruction issue (133 us for one expert each); behind the activation by
// instruction issue (7946 x 14336, MXFP4 H128, values: 744 MB in 168 us, about 33
// instructions a value at 0.66 per scheduler and clock).
#pragma once

#include "experts.h"
#include "quant_kernel.cuh"

namespace fp4q {

// A warp's way from segments to chunks: 32 segments' codes and scale bytes.
struct WarpStage {
    uint4 codes[32];
    uint32_t scales[32];
};

// Slot of chunk c (segment c / 4, part c % 4) in a buffer. Chunks 32 apart are
// 32 slots apart.
__device__ __forceinline__ int slot_of(int c) { return c ^ ((c >> 3) & 3); }

__device__ __forceinline__ void copy16(uint4* dst, const uint4* src, bool real)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src), "r"(real ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// Where this lane's segment lies: segment p of token (or taken row) i. one: the warp's 32
// segments all lie in the same row, so that addresses are a base of the warp plus the lane
// (a shuffle and a 64-bit product per chunk otherwise).
struct Place {
    uint32_t i, p;
    bool live, one;
};

// The places of a warp's tiles, a grid's step apart: the division is done once,
// a step adds its quotient and remainder. (Segment numbers and what a grid's
// step or two add to them stay below 2^32: the host checks.)
struct Places {
    uint32_t i0, p0, di, dp;  // row and segment of the warp's first lane; the step

    __device__ __forceinline__ Places(const RowQuantArgs& a, uint32_t s0, uint32_t step)
        : i0(s0 / a.spr), p0(s0 - i0 * a.spr), di(step / a.spr), dp(step - di * a.spr)
    {
    }
    __device__ __forceinline__ void next(const RowQuantArgs& a)
    {
        i0 += di;
        p0 += dp;
        if (p0 >= a.spr) {
            p0 -= a.spr;
            ++i0;
        }
    }
    __device__ __forceinline__ Place at(const RowQuantArgs& a, int lane) const
    {
        Place r{i0, p0 + lane, true, p0 + 32 <= a.spr};
        if (!r.one)  // a warp that spans rows
            while (r.p >= a.spr) {
                r.p -= a.spr;
                ++r.i;
            }
        r.live = r.i < a.n;
        return r;
    }
};

// The destination row of choice j of token i; -1 where there is none.
__device__ __forceinline__ int32_t row_of(const RowQuantArgs& a, int64_t i, int j)
{
    const int32_t r = a.slots == nullptr ? (int32_t)i : a.slots[i * a.k + j];
    return r < a.rows ? r : -1;
}

// One lane's quantized segment: its codes and scale bytes (block b at byte b).
struct Segment {
    uint4 q;
    uint32_t scales;
};

// process_segment with a lane's own variables as its output.
template <int B, int STRAT, int ROT>
__device__ __forceinline__ Segment quantize_segment(float (&y)[SEG], uint32_t keep,
                                                    const ScaleTables<STRAT>& tab)
{
    __align__(16) uint8_t codes[SEG / 2];
    __align__(4) uint8_t scales[4] = {};
    QuantArgs a;
    a.x = nullptr;
    a.n = 0;
    a.amax = nullptr;
    a.sg_out = nullptr;
    a.codes = codes;
    a.scales = scales;
    a.mse = nullptr;
    a.dq = nullptr;
    a.dq_kind = 0;
    a.keep = keep;
    a.mma_spr = 0;
    a.mma_atoms_k = 0;
    process_segment<B, STRAT, ROT>(y, 0, SEG, a, tab);
    Segment r;
    r.q = *reinterpret_cast<const uint4*>(codes);
    r.scales = *reinterpret_cast<const uint32_t*>(scales);
    return r;
}

template <int STRAT>
__device__ __forceinline__ float scale_value(const ScaleTables<STRAT>& tab, uint32_t byte)
{
    if constexpr (is_mx_strat(STRAT))
        return pow2f((int)byte - 127);
    else
        return tab.S[byte];
}

// Stores the warp's segments to the rows row(j), j < k, of each lane's segment
// (-1: none). All lanes take part.
template <int B, int STRAT, class Rows>
__device__ __forceinline__ void store_rows(const RowQuantArgs& a, const Segment& sg,
                                           WarpStage& st, const ScaleTables<STRAT>& tab,
                                           int lane, const Place& at, Rows row)
{
    constexpr int NB = SEG / B;      // blocks of a segment
    constexpr int QUAD = 4 / NB;     // segments of a 4-block group
    // Segments per row a multiple of QUAD: the groups of 4 blocks lie inside
    // the warp, and the first lane of each writes its 4 bytes at once.
    const bool whole = a.spr % QUAD == 0;
    uint32_t quad = sg.scales;
#pragma unroll
    for (int d = 1; d < QUAD; ++d)
        quad |= __shfl_down_sync(0xFFFFFFFFu, sg.scales, d) << (8 * NB * d);
    uint4 o[4];
    if (a.dq_kind == 2) {
        // bf16 values: chunk 32 c + lane is 8 values of segment 8 c + lane / 4
        st.codes[lane] = sg.q;
        st.scales[lane] = sg.scales;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t bytes = st.scales[8 * c + lane / 4];
            const float S = scale_value<STRAT>(tab, (bytes >> (8 * (lane % 4 * 8 / B))) & 0xFFu);
            float v[8];
            e2m1_unpack8(reinterpret_cast<const uint32_t*>(st.codes)[32 * c + lane], v);
            o[c].x = pack_bf16x2(__fmul_rn(v[0], S), __fmul_rn(v[1], S));
            o[c].y = pack_bf16x2(__fmul_rn(v[2], S), __fmul_rn(v[3], S));
            o[c].z = pack_bf16x2(__fmul_rn(v[4], S), __fmul_rn(v[5], S));
            o[c].w = pack_bf16x2(__fmul_rn(v[6], S), __fmul_rn(v[7], S));
        }
        __syncwarp();
    }
    for (int j = 0; j < a.k; ++j) {
        const int32_t r = row(j);
        const int64_t seg = (int64_t)r * a.spr + at.p;
        if (r >= 0) {
            reinterpret_cast<uint4*>(a.codes)[seg] = sg.q;
            const uint32_t kb = at.p * NB;
            uint8_t* dst = a.scales + ((int64_t)(r >> 7) * a.atoms_k + (kb >> 2)) * 512 +
                           16 * (r & 31) + 4 * ((r >> 5) & 3);
            if (whole) {
                if (lane % QUAD == 0)
                    *reinterpret_cast<uint32_t*>(dst) = quad;
            } else {
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    dst[(kb & 3) + b] = (uint8_t)(sg.scales >> (8 * b));
                if (at.p == a.spr - 1)  // padding blocks of the row's last group
                    for (uint32_t b = (kb & 3) + NB; b < 4; ++b)
                        dst[b] = 0;
            }
        }
        if (a.dq_kind == 2) {
            if (at.one) {
                if (r >= 0) {
                    uint4* dst = reinterpret_cast<uint4*>(a.dq) + (seg - lane) * 4 + lane;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        dst[32 * c] = o[c];
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int32_t rs = __shfl_sync(0xFFFFFFFFu, r, 8 * c + lane / 4);
                    const uint32_t ps = __shfl_sync(0xFFFFFFFFu, at.p, 8 * c + lane / 4);
                    if (rs >= 0)
                        reinterpret_cast<uint4*>(a.dq)[((int64_t)rs * a.spr + ps) * 4 + lane % 4] = o[c];
                }
            }
        } else if (a.dq_kind == 1 && r >= 0) {
            // fp32 values (for checks and calibration on small layers): each lane its segment
            float4* dst = reinterpret_cast<float4*>(a.dq) + seg * (SEG / 4);
            const uint32_t w[4] = {sg.q.x, sg.q.y, sg.q.z, sg.q.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float S = scale_value<STRAT>(tab, (sg.scales >> (8 * (c * 8 / B))) & 0xFFu);
                float v[8];
                e2m1_unpack8(w[c], v);
                dst[2 * c] = make_float4(__fmul_rn(v[0], S), __fmul_rn(v[1], S), __fmul_rn(v[2], S),
                                         __fmul_rn(v[3], S));
                dst[2 * c + 1] = make_float4(__fmul_rn(v[4], S), __fmul_rn(v[5], S), __fmul_rn(v[6], S),
                                             __fmul_rn(v[7], S));
            }
        }
    }
}

// The NVFP4 tables of a CTA (see ScaleTables), from the calibrated abs-max, or
// from the maxima of the abs-max pass's CTAs: every CTA joins them itself
// (no launch in between, no value to clear beforehand), and takes s_g as their maximum times
// fp32(1 / 2688), one product, where a calibrated abs-max is divided: what the header says of each. The
// product is a unit from the quotient for 22 maxima in a hundred (off by 0.81 of a unit at most,
// the quotient by 0.5), and codes that lie on a tie go with it. CTA 0 publishes s_g. Ends with a CTA barrier.
template <int STRAT>
__device__ __forceinline__ void row_scale_tables(const RowQuantArgs& a, ScaleTables<STRAT>& tab)
{
    if constexpr (!is_mx_strat(STRAT)) {
        static_assert(QTHREADS == 128, "one table entry a thread");
        __shared__ unsigned top[QTHREADS / 32];
        float sg;
        if (a.amax_parts == 0) {
            sg = global_scale_of(*a.amax);
        } else {
            unsigned m = 0;
            for (int i = threadIdx.x; i < a.amax_parts; i += QTHREADS)
                m = max(m, __float_as_uint(a.amax[i]));
            m = __reduce_max_sync(0xFFFFFFFFu, m);
            if (threadIdx.x % 32 == 0)
                top[threadIdx.x / 32] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < QTHREADS / 32; ++w)
                m = max(m, top[w]);
            sg = __fmul_rn(__uint_as_float(m), 1.0f / 2688.0f);
            sg = sg > 0.0f && sg <= FLT_MAX ? sg : 1.0f;
        }
        const int c = threadIdx.x;
        const float S = c <= 0x7E ? __fmul_rn(e4m3_dec((uint32_t)c), sg) : 0.0f;
        tab.S[c] = S;
        tab.R[c] = S == 0.0f ? 0.0f : guarded_rcp(S);
        if (c == 0) {
            tab.k = nv_consts(sg);
            if (blockIdx.x == 0)
                *a.sg_out = sg;
        }
        __syncthreads();
    }
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

// CTAs per SM that the registers are held to: searches as the compiler likes,
// else 4 (16384 x 8192 to two experts each, 4-over-6: 182 us; 5: 186, 6: 205; behind the
// activation, 8192 x 14336 MXFP4 H128: 184, 5 spills: 200, 3: 197).
template <int STRAT>
struct RowMinBlocks {
    static constexpr int value = STRAT == K_BRUTE_FORCE || STRAT == K_MX_BRUTE ? 1 : 4;
};

// ---------------------------------------------------------------- tokens

// Starts the copies of the warp's 32 segments from segment s0 of x.
__device__ __forceinline__ void fetch_tokens(const RowQuantArgs& a, uint32_t s0, int lane, uint4* in)
{
    const uint4* x4 = reinterpret_cast<const uint4*>(a.x) + (uint64_t)s0 * 4 + lane;
    uint4* dst = in + slot_of(lane);
    if (s0 + 32 <= a.nseg) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            copy16(dst + 32 * c, x4 + 32 * c, true);
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const bool real = s0 + 8 * c + lane / 4 < a.nseg;
            copy16(dst + 32 * c, real ? x4 + 32 * c : reinterpret_cast<const uint4*>(a.x), real);
        }
    }
}

// Segment s of x is segment s % spr of token s / spr. Persistent CTAs.
template <int B, int ROT, int STRAT>
__global__ void __launch_bounds__(QTHREADS, RowMinBlocks<STRAT>::value)
    token_quant_kernel(RowQuantArgs a, uint32_t ntiles)
{
    pdl_begin();
    __shared__ ScaleTables<STRAT> tab;
    __shared__ WarpStage stage[QTHREADS / 32];
    __shared__ uint4 inputs[QTHREADS / 32][2][32 * 4];
    const int lane = threadIdx.x & 31;
    WarpStage& st = stage[threadIdx.x / 32];
    uint4 (*in)[32 * 4] = inputs[threadIdx.x / 32];
    const uint32_t step = gridDim.x * QTHREADS;
    uint32_t s0 = blockIdx.x * QTHREADS + (threadIdx.x & ~31u);  // the warp's first segment
    fetch_tokens(a, s0, lane, in[0]);
    copies_commit();
    row_scale_tables<STRAT>(a, tab);
    Places places(a, s0, step);
    int buf = 0;
    for (uint32_t t = blockIdx.x; t < ntiles; t += gridDim.x, buf ^= 1, places.next(a)) {
        s0 += step;
        if (t + gridDim.x < ntiles)
            fetch_tokens(a, s0, lane, in[buf ^ 1]);
        copies_commit();
        copies_wait_but_one();
        __syncwarp();
        if (places.i0 < a.n) {  // warp-uniform
            const Place at = places.at(a, lane);
            // the rows of the first 32 choices, one a lane, on their way during the arithmetic
            int32_t mine = -1;
            if (at.one && lane < a.k)
                mine = row_of(a, at.i, lane);
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = in[buf][slot_of(4 * lane + k)];
            float y[SEG];
            unpack_seg<!is_mx_strat(STRAT)>(v, y);
            rotate_seg<ROT, !foldable<ROT, STRAT>()>(y, lane);
            const Segment sg = quantize_segment<B, STRAT, ROT>(y, a.keep, tab);
            store_rows<B, STRAT>(a, sg, st, tab, lane, at, [&](int j) {
                if (at.one && j < 32)
                    return __shfl_sync(0xFFFFFFFFu, mine, j);
                return at.live ? row_of(a, at.i, j) : -1;
            });
        }
        __syncwarp();
    }
}

// ---------------------------------------------------------------- gated activation

// The fp32 evaluation of v = g u sigmoid(z) and the relative error E that bounds it.
//
// v = (g u) / (1 + 2^a), a = -z log2 e, with the hardware's 2^x and 1/x: 2^x is off by 2
// units (2^-22) and its argument by 2^-23.4 |z| (product and constant), both times
// the share of 2^a in the sum, which is small where z > 0;
// the sum, the reciprocal (1 unit), two products and the ends of the bracket add
// 6 half units, 2^-21.4; gelu's z itself is off by 2^-21.7 |z|. With c = 2^-23 (silu) or
// 2^-21 (gelu) for each unit of |z| and |z| <= (z^2 + 1) / 2, E = 2^-20.4 + c/2 + c/2 z^2
// covers all of it (written in a^2 = z^2 log2(e)^2). The ends v (1 -+ E) of the bracket round
// to the same bf16 in all but about one value in three thousand.
template <int ACT>
struct GluError {
    static constexpr float half = ACT == FP4Q_ACT_GELU_TANH ? 0x1p-22f : 0x1p-24f;
    static constexpr float base = 0x1.85p-21f + half;
    static constexpr float square = half * 0.4805f;  // 1 / log2(e)^2 = 0.48045...
};

// g u sigmoid(z) in 64 bits by the library's functions, for what lies far out
// (a call: hardly ever taken, so it holds no registers elsewhere).
static __device__ __noinline__ double glu_far(double gu, double z) { return gu / (1.0 + exp(-z)); }

// h = bf16(fp32(g u sigmoid(z))) from its real value: 64 bits, one rounding to
// fp32, one to bf16. For values whose rounding the fp32 evaluation leaves open.
// In its range (lim) e^-z = 2^n e^f, |f| <= ln 2 / 2, by e^f's Taylor polynomial of degree 13
// (remainder below 2^-58), the quotient by Newton steps from the fp32
// reciprocal: off by 2^-48 at most (the argument reduction at |z| = 60; 2^-51 near 0). Outside of
// it by the library's exp and division.
template <int ACT>
__device__ __forceinline__ uint32_t glu_exact(float gf, float uf, bool lim)
{
    const double g = (double)gf, u = (double)uf;
    const double z = ACT == FP4Q_ACT_GELU_TANH ? 1.5957691216057307612 * (g + 0.044715 * g * g * g) : g;
    double h;
    if (lim && z < 600.0) {
        const double n = rint(z * -1.4426950408889634074);
        const double f = __fma_rn(n, -0.69314718055994530942, -z);
        constexpr double c[14] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040,
                                  1.0 / 40320, 1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800, 1.0 / 479001600,
                                  1.0 / 6227020800.0};
        double e = c[13];
#pragma unroll
        for (int k = 12; k >= 0; --k)
            e = __fma_rn(e, f, c[k]);
        const double q = 1.0 + e * __longlong_as_double((long long)((int)n + 1023) << 52);
        double r = (double)__frcp_rn((float)q);
        r = __fma_rn(r, __fma_rn(-q, r, 1.0), r);
        r = __fma_rn(r, __fma_rn(-q, r, 1.0), r);
        h = g * u * r;
    } else {
        h = glu_far(g * u, z);
    }
    return __bfloat16_as_ushort(__float2bfloat16_rn((float)h));
}

// The range in which E holds: z > -60 keeps 2^a and its reciprocal in range,
// |v| > 2^-100 the products (g u and v differ by a factor below 2^88).
constexpr float GLU_Z = -60.0f, GLU_V = 0x1p-100f;

// One value again, alone: the fp32 evaluation if it decides, else 64 bits.
template <int ACT>
__device__ __forceinline__ uint32_t glu_one(uint32_t gb, uint32_t ub)
{
    if ((gb << 1) == 0 || (ub << 1) == 0)
        return ((gb ^ ub) & 0x80000000u) >> 16;  // a zero factor gives a signed zero
    const float g = __uint_as_float(gb), u = __uint_as_float(ub);
    float z = g;
    if constexpr (ACT == FP4Q_ACT_GELU_TANH)
        z = (g * 1.5957691216f) * __fmaf_rn(g * 0.044715f, g, 1.0f);
    const float a = z * -1.4426950409f;
    float t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(a));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t + 1.0f));
    const float v = (g * u) * r;
    const float d = v * __fmaf_rn(a * a, GluError<ACT>::square, GluError<ACT>::base);
    const bool lim = z > GLU_Z && fabsf(v) > GLU_V;
    const uint32_t hi = __bfloat16_as_ushort(__float2bfloat16_rn(v + d));
    if (lim && __bfloat16_as_ushort(__float2bfloat16_rn(v - d)) == hi)
        return hi;
    return glu_exact<ACT>(g, u, lim);
}

// Two values of h as packed bf16, from packed bf16 gates and values (packed fp32
// operations). Pair I's bit is set in open where the bracket's ends differ; zmin and
// vmin collect the smallest z and |v|.
template <int ACT, int I>
__device__ __forceinline__ uint32_t glu_pair(uint32_t g2, uint32_t u2, uint32_t& open, float& zmin,
                                             float& vmin)
{
    const f32x2 g = pk2(bf_lo(g2), bf_hi<true>(g2)), u = pk2(bf_lo(u2), bf_hi<true>(u2));
    f32x2 z = g;
    if constexpr (ACT == FP4Q_ACT_GELU_TANH)
        z = mul2(mul2(g, pk2(1.5957691216f, 1.5957691216f)),
                 fma2(mul2(g, pk2(0.044715f, 0.044715f)), g, pk2(1.0f, 1.0f)));
    const f32x2 a = mul2(z, pk2(-1.4426950409f, -1.4426950409f));
    float z0, z1, t0, t1, r0, r1;
    upk2(a, t0, t1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t0) : "f"(t0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t1) : "f"(t1));
    upk2(add2(pk2(t0, t1), pk2(1.0f, 1.0f)), t0, t1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(t0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(t1));
    const f32x2 v = mul2(mul2(g, u), pk2(r0, r1));
    constexpr float base = GluError<ACT>::base, square = GluError<ACT>::square;
    const f32x2 d = mul2(v, fma2(mul2(a, a), pk2(square, square), pk2(base, base)));
    float lo0, lo1, hi0, hi1, v0, v1;
    upk2(add2(v, d), hi0, hi1);
    upk2(sub2(v, d), lo0, lo1);
    upk2(v, v0, v1);
    upk2(z, z0, z1);
    zmin = fminf(fminf(zmin, z0), z1);
    vmin = fminf(fminf(vmin, fabsf(v0)), fabsf(v1));
    const uint32_t hi = pack_bf16x2(hi0, hi1);
    if (pack_bf16x2(lo0, lo1) != hi)
        open |= 1u << I;
    return hi;
}

// This lane's segment of h, widened, from its gates and values in shared memory. The pairs
// run without a branch between them; the undecided ones follow one by one, patched through
// the gates' slots.
template <int ACT>
__device__ __forceinline__ void glu_segment(uint4* gate, const uint4* value, int lane, float (&y)[SEG])
{
    uint4 h[4];
    uint32_t open = 0;
    float zmin = 0.0f, vmin = 1.0f;
    static_for<4>([&](auto kc) {
        constexpr int k = decltype(kc)::value;
        const uint4 g = gate[slot_of(4 * lane + k)], u = value[slot_of(4 * lane + k)];
        h[k].x = glu_pair<ACT, 4 * k>(g.x, u.x, open, zmin, vmin);
        h[k].y = glu_pair<ACT, 4 * k + 1>(g.y, u.y, open, zmin, vmin);
        h[k].z = glu_pair<ACT, 4 * k + 2>(g.z, u.z, open, zmin, vmin);
        h[k].w = glu_pair<ACT, 4 * k + 3>(g.w, u.w, open, zmin, vmin);
    });
    // (an infinite v, as of an overflowing g u, has a bracket that ends in NaN: open)
    if (!(zmin > GLU_Z && vmin > GLU_V))
        open = 0xFFFFu;
    if (open != 0) {
        uint32_t* gw = reinterpret_cast<uint32_t*>(gate);
        const uint32_t* uw = reinterpret_cast<const uint32_t*>(value);
        for (uint32_t m = open; m != 0; m &= m - 1) {
            const int pair = __ffs(m) - 1;
            const int at = slot_of(4 * lane + pair / 4) * 4 + pair % 4;
            uint32_t g2 = gw[at], u2 = uw[at], out = 0;
#pragma unroll 1
            for (int k = 0; k < 2; ++k, g2 >>= 16, u2 >>= 16)
                out = (out >> 16) | (glu_one<ACT>(g2 << 16, u2 << 16) << 16);
            gw[at] = out;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint4 w = gate[slot_of(4 * lane + k)];
            h[k].x = open & (1u << (4 * k)) ? w.x : h[k].x;
            h[k].y = open & (2u << (4 * k)) ? w.y : h[k].y;
            h[k].z = open & (4u << (4 * k)) ? w.z : h[k].z;
            h[k].w = open & (8u << (4 * k)) ? w.w : h[k].w;
        }
    }
    unpack_seg<true>(h, y);
}

// Starts the copies of the warp's 32 segments of gate and value. row: the
// row of this lane's segment, -1 for none (zeros).
__device__ __forceinline__ void fetch_glu(const RowQuantArgs& a, const Place& at, int32_t row, int lane,
                                          uint4 (*in)[32 * 4])
{
    const uint4* x4 = reinterpret_cast<const uint4*>(a.x);
    uint4* gate = in[0] + slot_of(lane);
    uint4* value = in[1] + slot_of(lane);
    if (at.one && row >= 0) {
        const uint4* g = x4 + ((int64_t)row * 2 * a.spr + (at.p - lane)) * 4 + lane;
        const uint4* u = g + (int64_t)a.spr * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            copy16(gate + 32 * c, g + 32 * c, true);
            copy16(value + 32 * c, u + 32 * c, true);
        }
    } else {
        // (of a warp whose row is one and not there, every lane comes here)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int32_t r = __shfl_sync(0xFFFFFFFFu, row, 8 * c + lane / 4);
            const uint32_t p = __shfl_sync(0xFFFFFFFFu, at.p, 8 * c + lane / 4);
            const uint4* g = x4 + (r >= 0 ? ((int64_t)r * 2 * a.spr + p) * 4 + lane % 4 : 0);
            copy16(gate + 32 * c, g, r >= 0);
            copy16(value + 32 * c, g + (r >= 0 ? (int64_t)a.spr * 4 : 0), r >= 0);
        }
    }
}

// Walks a warp over its tiles of taken rows: the copies of the next tile are in flight, and
// the row numbers of the one after it, while body(y, place, row) works on the current one.
template <int ACT, class Body>
__device__ __forceinline__ void glu_tiles(const RowQuantArgs& a, uint32_t ntiles, int lane,
                                          uint4 (*in)[2][32 * 4], Body body)
{
    auto row_at = [&](const Place& at) { return at.live ? row_of(a, at.i, 0) : -1; };
    Places places(a, blockIdx.x * QTHREADS + (threadIdx.x & ~31u), gridDim.x * QTHREADS);
    Place now = places.at(a, lane);
    int32_t row = row_at(now);
    fetch_glu(a, now, row, lane, in[0]);
    copies_commit();
    places.next(a);
    Place next = places.at(a, lane);  // (past the last tile: not live, no row, no copy)
    int32_t next_row = row_at(next);
    int buf = 0;
    for (uint32_t t = blockIdx.x; t < ntiles; t += gridDim.x, buf ^= 1) {
        if (t + gridDim.x < ntiles)
            fetch_glu(a, next, next_row, lane, in[buf ^ 1]);
        copies_commit();
        places.next(a);
        const Place then = places.at(a, lane);
        const int32_t then_row = row_at(then);
        copies_wait_but_one();
        __syncwarp();
        if (__any_sync(0xFFFFFFFFu, now.live)) {
            float y[SEG];
            glu_segment<ACT>(in[buf][0], in[buf][1], lane, y);
            body(y, now, row);
        }
        __syncwarp();
        now = next;
        row = next_row;
        next = then;
        next_row = then_row;
    }
}

template <int B, int ROT, int STRAT, int ACT>
__global__ void __launch_bounds__(QTHREADS, RowMinBlocks<STRAT>::value)
    glu_quant_kernel(RowQuantArgs a, uint32_t ntiles)
{
    pdl_begin();
    __shared__ ScaleTables<STRAT> tab;
    __shared__ WarpStage stage[QTHREADS / 32];
    __shared__ uint4 inputs[QTHREADS / 32][2][2][32 * 4];
    const int lane = threadIdx.x & 31;
    WarpStage& st = stage[threadIdx.x / 32];
    row_scale_tables<STRAT>(a, tab);
    glu_tiles<ACT>(a, ntiles, lane, inputs[threadIdx.x / 32], [&](float (&y)[SEG], const Place& at, int32_t row) {
        rotate_seg<ROT, !foldable<ROT, STRAT>()>(y, lane);
        const Segment sg = quantize_segment<B, STRAT, ROT>(y, a.keep, tab);
        store_rows<B, STRAT>(a, sg, st, tab, lane, at, [&](int) { return row; });
    });
}

// Resident CTAs per SM of one kernel (a template value, so that each kernel
// keeps its own), queried once per process; -1 if the query fails.
template <auto KERNEL>
int resident_rows()
{
    static std::atomic<int> per_sm{0};
    int n = per_sm.load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERNEL, QTHREADS, 0) != cudaSuccess)
            return -1;
        n = n < 1 ? 1 : n;
        per_sm.store(n, std::memory_order_relaxed);
    }
    return n;
}

// Launch of a row quantize kernel over the resident CTAs, at most `most` (then
// as many on every SM); their number goes to *ctas.
template <auto KERNEL>
cudaError_t launch_rows(const RowQuantArgs& a, cudaStream_t st, int64_t most = 0x7FFFFFFF,
                        int* ctas = nullptr)
{
    const int64_t nblk = ((int64_t)a.nseg + QTHREADS - 1) / QTHREADS;
    int dev = 0, sms = 0;
    int64_t per_sm = resident_rows<KERNEL>();
    if (per_sm < 0 || cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms > most)
        return cudaErrorUnknown;
    if (per_sm * sms > most)
        per_sm = most / sms;
    const int64_t grid = nblk < per_sm * sms ? nblk : per_sm * sms;
    if (ctas != nullptr)
        *ctas = (int)grid;
    return launch_pdl(KERNEL, dim3((unsigned)grid), dim3(QTHREADS), 0, st, a, (uint32_t)nblk);
}

#define FP4Q_ROWS_CASE(KERNEL_, B_, S_, R_) \
    if (strat == S_ && rot == R_)           \
        return launch_rows<KERNEL_<B_, R_, S_>>(a, st);
#define FP4Q_ROWS_ROTS(KERNEL_, B_, S_)  \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 0)   \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 16)  \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 32)  \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 64)  \
    FP4Q_ROWS_CASE(KERNEL_, B_, S_, 128)
#define FP4Q_GLU_CASE(B_, S_, R_)                                                        \
    if (strat == S_ && rot == R_)                                                        \
        return a.act == FP4Q_ACT_SILU                                                    \
                   ? launch_rows<glu_quant_kernel<B_, R_, S_, FP4Q_ACT_SILU>>(a, st)     \
                   : launch_rows<glu_quant_kernel<B_, R_, S_, FP4Q_ACT_GELU_TANH>>(a, st);
#define FP4Q_GLU_ROTS(B_, S_)  \
    FP4Q_GLU_CASE(B_, S_, 0)   \
    FP4Q_GLU_CASE(B_, S_, 16)  \
    FP4Q_GLU_CASE(B_, S_, 32)  \
    FP4Q_GLU_CASE(B_, S_, 64)  \
    FP4Q_GLU_CASE(B_, S_, 128)

}  // namespace fp4q

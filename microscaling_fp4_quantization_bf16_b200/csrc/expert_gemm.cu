// expert_gemm.cu -- grouped W4A4 product on the block-scaled tensor cores.
//
//   d[r, m] = alpha_e sum_k a[r, k] w[e, m, k]   for the rows r of expert e
//
// The weights are the MMA's A operand (128 rows of w, the lanes of the
// accumulator) and the tokens its B operand (up to TN rows of a, its columns):
// the number of columns of one MMA can follow the number of rows that an
// expert really has (a multiple of 16), the number of lanes cannot, and an
// expert at decode time has a few rows only.
//
// One CTA per SM walks tiles of 128 outputs x TN rows (static, persistent).
// Warp 0 brings in the operands: per 256 values of k, both codes by TMA
// (128-byte rows, 128-byte swizzle) and their scale bytes, which lie in 512-byte
// atoms of 128 rows x 4 blocks in global memory already, by bulk copies. Warp 1
// copies the scale atoms into TMEM (tcgen05.cp, 32 rows x 16 bytes repeated over the four lane
// quarters) and issues the MMAs, 64 values of k each; both run in order in the
// tensor pipe, so the TMEM columns of the scales need no second buffer. Warps 2..5
// read the finished accumulator, scale it by alpha and store.
//
// The accumulator is double buffered, so a tile's stores run beside the next
// tile's products. At TN = 256 two of them and 48 columns of scales do not fit
// the 512 columns: the second starts at column 208, and the MMA waits only until
// the 48 columns that both share have been read.
//
// Waits are bounded: one that runs out raises the CTA's abort flag and the
// device error counter, and every role leaves after its copies have landed.
#include "experts.h"
#include "fp4q_device.cuh"

namespace fp4q {

namespace {

constexpr int GTHREADS = 192;
constexpr int CHUNK = 256;                 // values of k per stage: 128 bytes of codes
constexpr int WROWS = 128;                 // outputs of a tile
constexpr int ATOM = 512;                  // bytes of 128 rows x 4 block scales
constexpr uint32_t POLLS = 1u << 22;       // of a wait before it gives up
constexpr int SMEM_LIMIT = 227 * 1024;
constexpr int ALIGN_SLACK = 1024;

template <int TN>
struct Tile {
    static constexpr int BOX = TN == 128 ? 32 : 64;              // rows of one token box
    static constexpr int WBYTES = WROWS * 128;
    static constexpr int ABYTES = TN * 128;
    static constexpr int SW = 4 * ATOM;                          // weight scales of a stage
    static constexpr int SA = 4 * ATOM * (TN / 128);             // token scales
    static constexpr int STAGE = WBYTES + ABYTES + SW + SA;
    // barriers, prefix sums of the experts' tiles, abort flag and TMEM address
    static constexpr int FIXED = 256 + (FP4Q_MAX_EXPERTS + 1) * 4 + 64;
    static constexpr int STAGES = (SMEM_LIMIT - ALIGN_SLACK - FIXED) / STAGE > 10
                                      ? 10
                                      : (SMEM_LIMIT - ALIGN_SLACK - FIXED) / STAGE;
    static constexpr int SMEM = STAGES * STAGE + FIXED + ALIGN_SLACK;
    // TMEM columns: two accumulators (overlapping at TN = 256), then the scales
    static constexpr int SHARE = TN == 256 ? 48 : 0;
    static constexpr int SECOND = TN - SHARE;                    // first column of buffer 1
    static constexpr int COL_SW = 2 * TN - SHARE;                // 16 columns
    static constexpr int COL_SA = COL_SW + 16;                   // 16 per 128 rows
    static constexpr int COLS = 512;
    static_assert(TN == 128 || TN == 256, "row tiles start at a scale atom");
    static_assert(COL_SA + 16 * (TN / 128) <= COLS, "TMEM");
    static_assert(STAGES >= 3, "stages");
};

__device__ __forceinline__ uint32_t sptr(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool bar_poll(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// False when the wait ran out or another role of the CTA has given up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag)
{
    for (uint32_t i = 0; i < POLLS; ++i) {
        if (bar_poll(bar, parity))
            return true;
        if (*abort_flag)
            return false;
    }
    *abort_flag = 1;
    return false;
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
        : "memory");
}

// Shared-memory matrix descriptors (start address, leading and stride byte
// offsets in 16-byte units, descriptor version 1 in bits 46-47, swizzle in bits 61-63).
// Codes: K-major rows of 128 bytes, 128-byte swizzle (2), 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_codes(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Scale atoms: 32 rows of 16 bytes, no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) |
           ((uint64_t)1 << 46);
}

__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <bool NV>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                    uint32_t sb, uint32_t accumulate)
{
    if constexpr (NV)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X"
            " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
            : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
          "=r"(v[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Walks the CTA's tiles: tile number -> expert, first output, first row, rows.
// Experts in order; within one, the row tiles of the same outputs are neighbours, so that
// CTAs running together share the weights.
template <int TN>
struct Walk {
    const int32_t* prefix;  // shared: token tiles of the experts before e
    int experts, wtiles, e;
    int64_t total;

    __device__ __forceinline__ Walk(const int32_t* p, int ex, int wt)
        : prefix(p), experts(ex), wtiles(wt), e(0), total((int64_t)p[ex] * wt)
    {
    }
    __device__ __forceinline__ void at(int64_t item, int& wtile, int& ttile)
    {
        while (item >= (int64_t)prefix[e + 1] * wtiles)
            ++e;
        const int tt = prefix[e + 1] - prefix[e];
        const int idx = (int)(item - (int64_t)prefix[e] * wtiles);
        wtile = idx / tt;
        ttile = idx - wtile * tt;
    }
};

template <int TN, bool NV, bool F32>
__global__ void __launch_bounds__(GTHREADS, 1)
    expert_gemm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                       ExpertGemmArgs p)
{
    using T = Tile<TN>;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(raw_smem) + ALIGN_SLACK - 1) & ~uintptr_t(ALIGN_SLACK - 1));
    uint8_t* fixed = smem + T::STAGES * T::STAGE;
    const uint32_t bars = sptr(fixed);
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (T::STAGES + s); };
    auto acc_full = [&](int b) { return bars + 8 * (2 * T::STAGES + b); };
    auto acc_free = [&](int b) { return bars + 8 * (2 * T::STAGES + 2 + b); };
    static_assert(8 * (2 * T::STAGES + 4) <= 256, "barriers");
    int32_t* prefix = reinterpret_cast<int32_t*>(fixed + 256);
    volatile int* abort_flag = reinterpret_cast<int*>(fixed + 256 + (FP4Q_MAX_EXPERTS + 1) * 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fixed + 256 + (FP4Q_MAX_EXPERTS + 1) * 4 + 4);

    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < T::STAGES; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), 1);
            bar_init(acc_free(b), 4);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sptr(tmem_slot)),
                     "r"((uint32_t)T::COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_begin();
    if (warp == 0) {
        // token tiles of the experts before each; segments outside the buffer count none
        int carry = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            int t = 0;
            if (e < p.experts) {
                const int64_t c = p.counts[e], s = p.starts[e];
                if (c > 0 && s >= 0 && s % kSegRows == 0 && s + c <= p.rows)
                    t = (int)((c + TN - 1) / TN);
            }
            int inc = t;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                inc += lane >= d ? v : 0;
            }
            if (e < p.experts)
                prefix[e + 1] = carry + inc;
            carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
        if (lane == 0)
            prefix[0] = 0;
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;

    const int wtiles = (p.N + WROWS - 1) / WROWS;
    const int chunks = (p.K + CHUNK - 1) / CHUNK;
    constexpr int APC = NV ? 4 : 2;                         // scale atoms of a chunk
    const int atoms = NV ? (p.K + 63) / 64 : (p.K + 127) / 128;  // along a row
    Walk<TN> walk(prefix, p.experts, wtiles);

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int64_t item = blockIdx.x; ok && item < walk.total; item += gridDim.x) {
                int wt, tt;
                walk.at(item, wt, tt);
                const int row0 = p.starts[walk.e] + tt * TN;
                const int valid = min(TN, p.counts[walk.e] - tt * TN);
                const int boxes = (valid + T::BOX - 1) / T::BOX;
                const int groups = (valid + 127) / 128;  // scale atoms along the rows
                const int64_t wrow = (int64_t)walk.e * p.N + wt * WROWS;
                const uint8_t* ws = p.w_scales + ((int64_t)walk.e * wtiles + wt) * atoms * ATOM;
                const uint8_t* as = p.a_scales + (int64_t)(row0 / 128) * atoms * ATOM;
                for (int c = 0; c < chunks; ++c, ++it) {
                    const int s = it % T::STAGES;
                    if (it >= T::STAGES && !bar_wait(empty(s), ((it / T::STAGES) & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t* st = smem + s * T::STAGE;
                    const uint32_t n = ATOM * min(APC, atoms - c * APC);
                    bar_expect(full(s), T::WBYTES + boxes * T::BOX * 128 + n * (1 + groups));
                    tma_box(sptr(st), &wmap, c * 128, (int)wrow, full(s));
                    for (int b = 0; b < boxes; ++b)
                        tma_box(sptr(st + T::WBYTES + b * T::BOX * 128), &amap, c * 128, row0 + b * T::BOX,
                                full(s));
                    uint8_t* sc = st + T::WBYTES + T::ABYTES;
                    bulk_load(sptr(sc), ws + (int64_t)c * APC * ATOM, n, full(s));
                    for (int g = 0; g < groups; ++g)
                        bulk_load(sptr(sc + T::SW + g * 4 * ATOM), as + ((int64_t)g * atoms + c * APC) * ATOM,
                                  n, full(s));
                }
            }
            if (!ok) {
                atomicAdd(p.err, 1u);
                // copies in flight land before the CTA gives its memory back
                for (int j = it < T::STAGES ? 0 : it - T::STAGES; j < it; ++j)
                    for (uint32_t i = 0; i < POLLS && !bar_poll(full(j % T::STAGES), (j / T::STAGES) & 1); ++i)
                        ;
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0, tile = 0;
            bool ok = true;
            for (int64_t item = blockIdx.x; ok && item < walk.total; item += gridDim.x, ++tile) {
                int wt, tt;
                walk.at(item, wt, tt);
                const int valid = min(TN, p.counts[walk.e] - tt * TN);
                const int cols = (valid + 15) & ~15;
                const int groups = (valid + 127) / 128;
                const int buf = tile & 1;
                // buffers apart: tile - 2 has been read; overlapping: the shared
                // columns of tile - 1 have
                if (T::SHARE > 0 ? tile >= 1 : tile >= 2) {
                    const int b = T::SHARE > 0 ? buf ^ 1 : buf;
                    const int phase = T::SHARE > 0 ? (tile - 1) / 2 : (tile - 2) / 2;
                    if (!bar_wait(acc_free(b), phase & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t d = tmem + buf * T::SECOND;
                // instruction descriptor: E2M1 x E2M1, columns / 8 at bit 17, scale type (0 E4M3,
                // 1 E8M0) at bit 23, rows / 16 at bit 24; scale byte pair of MXFP4 at bits 4 and 29
                const uint32_t idesc = (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) |
                                       ((NV ? 0u : 1u) << 23) | ((WROWS >> 4) << 24);
                for (int c = 0; c < chunks; ++c, ++it) {
                    const int s = it % T::STAGES;
                    if (!bar_wait(full(s), (it / T::STAGES) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t st = sptr(smem + s * T::STAGE);
                    const uint32_t sc = st + T::WBYTES + T::ABYTES;
                    const int na = min(APC, atoms - c * APC);
                    for (int k = 0; k < na; ++k) {
                        copy_scales(tmem + T::COL_SW + 4 * k, desc_scales(sc + k * ATOM));
                        for (int g = 0; g < groups; ++g)
                            copy_scales(tmem + T::COL_SA + 4 * (TN / 128) * k + 4 * g,
                                        desc_scales(sc + T::SW + g * 4 * ATOM + k * ATOM));
                    }
                    const int steps = min(CHUNK / 64, (p.K - c * CHUNK + 63) / 64);
                    const uint64_t da = desc_codes(st), db = desc_codes(st + T::WBYTES);
                    for (int k = 0; k < steps; ++k) {
                        const int a = NV ? k : k / 2;            // scale atom of this step
                        const uint32_t id = NV ? 0u : 2u * (k & 1);  // its byte pair
                        mma<NV>(d, da + 2 * k, db + 2 * k, idesc | (id << 4) | (id << 29),
                                tmem + T::COL_SW + 4 * a, tmem + T::COL_SA + 4 * (TN / 128) * a,
                                (c | k) != 0);
                    }
                    commit(empty(s));
                }
                if (ok)
                    commit(acc_full(buf));
            }
            if (!ok)
                atomicAdd(p.err, 1u);
        }
    } else {
        const int quarter = warp & 3;  // TMEM lanes 32 quarter .. + 31
        int tile = 0;
        bool ok = true;
        for (int64_t item = blockIdx.x; ok && item < walk.total; item += gridDim.x, ++tile) {
            int wt, tt;
            walk.at(item, wt, tt);
            const int row0 = p.starts[walk.e] + tt * TN;
            const int valid = min(TN, p.counts[walk.e] - tt * TN);
            const int buf = tile & 1;
            const float alpha = NV ? __fmul_rn(*p.a_sg, p.w_sg[walk.e]) : 1.0f;
            if (!__all_sync(0xFFFFFFFFu, bar_wait(acc_full(buf), (tile / 2) & 1, abort_flag))) {
                ok = false;
                break;
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t acc = tmem + ((uint32_t)(32 * quarter) << 16) + buf * T::SECOND;
            const int m = wt * WROWS + 32 * quarter + lane;
            const bool mine = m < p.N;
            auto store = [&](int col, uint32_t bits) {
                if (mine && col < valid) {
                    const float v = __fmul_rn(__uint_as_float(bits), alpha);
                    const int64_t at = (int64_t)(row0 + col) * p.N + m;
                    if constexpr (F32)
                        static_cast<float*>(p.d)[at] = v;
                    else
                        static_cast<__nv_bfloat16*>(p.d)[at] = __float2bfloat16_rn(v);
                }
            };
            auto release = [&]() {
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    bar_arrive(acc_free(buf));
            };
            auto part16 = [&](int col, bool last) {
                uint32_t v[16];
                tmem_load16(acc + col, v);
                if (last)
                    release();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    store(col + i, v[i]);
            };
            if constexpr (T::SHARE > 0) {
                // the columns that the other buffer shares come first
                const int first = buf == 0 ? TN - T::SHARE : 0;
                for (int col = first; col < first + T::SHARE; col += 16)
                    part16(col, col + 16 == first + T::SHARE);
                const int lo = buf == 0 ? 0 : T::SHARE;
                for (int col = lo; col < lo + TN - T::SHARE && col < valid; col += 16)
                    part16(col, false);
            } else {
                for (int col = 0; col < valid; col += 16)
                    part16(col, col + 16 >= valid);
            }
        }
        if (!ok && lane == 0)
            atomicAdd(p.err, 1u);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)T::COLS));
    }
}

template <int TN, bool NV, bool F32>
cudaError_t gemm_one(const CUtensorMap& wmap, const uint8_t* a_codes, const ExpertGemmArgs& a, int sms,
                     cudaStream_t st)
{
    CUtensorMap amap;
    if (!make_byte_map(&amap, a_codes, a.K / 2, a.rows, Tile<TN>::BOX))
        return cudaErrorInvalidValue;
    auto kern = expert_gemm_kernel<TN, NV, F32>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Tile<TN>::SMEM);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kern, dim3((unsigned)sms), dim3(GTHREADS), Tile<TN>::SMEM, st, wmap, amap, a);
}

template <int TN>
cudaError_t gemm_type(bool nv, bool out32, const CUtensorMap& wmap, const uint8_t* a_codes,
                      const ExpertGemmArgs& a, int sms, cudaStream_t st)
{
    if (nv)
        return out32 ? gemm_one<TN, true, true>(wmap, a_codes, a, sms, st)
                     : gemm_one<TN, true, false>(wmap, a_codes, a, sms, st);
    return out32 ? gemm_one<TN, false, true>(wmap, a_codes, a, sms, st)
                 : gemm_one<TN, false, false>(wmap, a_codes, a, sms, st);
}

}  // namespace

cudaError_t launch_expert_gemm(bool nv, bool out32, int64_t mean_rows, const uint8_t* a_codes,
                               const uint8_t* w_codes, const ExpertGemmArgs& a, cudaStream_t st)
{
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess)
        return e;
    CUtensorMap wmap;
    if (!make_byte_map(&wmap, w_codes, a.K / 2, (int64_t)a.experts * a.N, WROWS))
        return cudaErrorInvalidValue;
    if (mean_rows <= 128)
        return gemm_type<128>(nv, out32, wmap, a_codes, a, sms, st);
    return gemm_type<256>(nv, out32, wmap, a_codes, a, sms, st);
}

}  // namespace fp4q

// expert_gemm.cu -- grouped W4A4 product on the block-scaled tensor cores.
//
//   d[r, m] = alpha_e sum_k a[r, k] w[e, m, k]   for the rows r of expert e
//
// The weights are the MMA's A operand (the lanes of the accumulator) and the
// tokens its B operand (its columns): the number of columns of one MMA can follow
// the number of rows that an expert really has, the number of lanes cannot,
// and an expert at decode time has a few rows only.
//
// Two forms, by the mean rows of an expert that has any:
//  - up to 128: one CTA to a tile of 128 outputs x up to 128 rows. Bound by reading the
//    weights; six stages of loads in flight.
//  - above: two CTAs to a tile of 256 outputs x up to 256 rows (cta_group::2). Each
//    CTA brings in its own 128 outputs' weights and half of the tokens, and the MMA
//    reads both halves: 38 KB a CTA for 256 values of k, where a CTA alone would need 54. A single CTA
//    with 128 x 256 tiles was bound by that: 380 us for its loads alone (66 bytes a
//    clock and SM from L2), 443 us in all, on 16384 rows x 4096 x 14336, 8 experts, NVFP4.
//
// One CTA (or pair) per SM (two) walks the tiles (static, persistent).
// Warp 0 brings in the operands: per 256 values of k, both codes by TMA
// (128-byte rows, 128-byte swizzle) and their scale bytes, which lie in 512-byte
// atoms of 128 rows x 4 blocks in global memory already. Warp 1
// copies the scale atoms into TMEM (tcgen05.cp, 32 rows x 16 bytes repeated over the four lane
// quarters) and issues the MMAs, 64 values of k each; both run in order in the
// tensor pipe, so the TMEM columns of the scales need no second buffer. The whole warp walks
// the loop and one elected lane issues: these instructions take uniform registers, and behind a branch on
// the lane number each cost about 150 clocks (1062 us against 537 on the product above). Warps 2..5
// read the finished accumulator, scale it by alpha and store.
//
// The accumulator is double buffered, so a tile's stores run beside the next
// tile's products. At 256 columns two of them and 48 columns of scales do not fit
// the 512 columns: the second starts at column 208, and the MMA waits only until
// the 48 columns that both share have been read.
//
// Waits are bounded: one that runs out raises the CTA's abort flag and the
// device error counter, and every role leaves after its copies have landed and its
// products have ended.
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

template <bool PAIR>
struct Tile {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TN = PAIR ? 256 : 128;                  // most rows of a tile
    static constexpr int ROWS = TN / CTAS;                       // of which a CTA loads
    static constexpr int BOX = PAIR ? 128 : 32;                  // rows of one token box
    static constexpr int WBYTES = WROWS * 128;
    static constexpr int ABYTES = ROWS * 128;
    static constexpr int SW = 4 * ATOM;                          // weight scales of a stage
    static constexpr int SA = 4 * ATOM * (TN / 128);             // token scales
    static constexpr int STAGE = WBYTES + ABYTES + SW + SA;
    // barriers, prefix sums of the experts' tiles, abort flag and TMEM address
    static constexpr int FIXED = 256 + (FP4Q_MAX_EXPERTS + 1) * 4 + 64;
    static constexpr int STAGES = (SMEM_LIMIT - ALIGN_SLACK - FIXED) / STAGE;
    static constexpr int SMEM = STAGES * STAGE + FIXED + ALIGN_SLACK;
    // TMEM columns: two accumulators (overlapping at TN = 256), then the scales
    static constexpr int SHARE = TN == 256 ? 48 : 0;
    static constexpr int SECOND = TN - SHARE;                    // first column of buffer 1
    static constexpr int COL_SW = 2 * TN - SHARE;                // 16 columns
    static constexpr int COL_SA = COL_SW + 16;                   // 16 per 128 rows
    static constexpr int COLS = 512;
    static_assert(COL_SA + 16 * (TN / 128) <= COLS, "TMEM");
    static_assert(STAGES >= 4 && 8 * (2 * STAGES + 4) <= 256, "stages");
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

// Arrives on a barrier of the pair's first CTA (a cluster address).
__device__ __forceinline__ void bar_arrive_first(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool bar_poll(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// False when the wait ran out or another role of the CTA has given up. Lanes may see the
// two in another order: no warp barrier lies inside a loop that a lane leaves over this, and the
// lanes of a role agree once a tile. (A vote after each wait cost the large product 377 -> 405 us.)
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

// One box by TMA. PAIR: the barrier may be the other CTA's.
template <bool PAIR>
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    if constexpr (PAIR) {
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
        return;
    }
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

template <bool PAIR>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

#define FP4Q_MMA_ASM(GROUP_, KIND_)                                                  \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"                   \
                 "tcgen05.mma.cta_group::" GROUP_ ".kind::" KIND_                    \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                  \
                 "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)       \
                 : "memory")

template <bool PAIR, bool NV>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                    uint32_t sb, uint32_t accumulate)
{
    if constexpr (PAIR && NV)
        FP4Q_MMA_ASM("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (PAIR)
        FP4Q_MMA_ASM("2", "mxf4.block_scale.scale_vec::2X");
    else if constexpr (NV)
        FP4Q_MMA_ASM("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else
        FP4Q_MMA_ASM("1", "mxf4.block_scale.scale_vec::2X");
}
#undef FP4Q_MMA_ASM

// Arrives on the barrier (PAIR: of both CTAs) once everything issued so far has finished.
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
            " [%0], %1;" ::"r"(bar), "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}

// The same shared address in the pair's first CTA.
__device__ __forceinline__ uint32_t in_first(uint32_t addr)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
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

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t is;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(is));
    return is != 0;
}

// Walks the CTA's tiles: tile number -> expert, first output, first row, rows.
// Experts in order; within one, the row tiles of the same outputs are neighbours, so that
// CTAs running together share the weights.
struct Walk {
    const int32_t* prefix;  // shared: token tiles of the experts before e
    int experts, wtiles, e;
    int64_t total;

    __device__ __forceinline__ Walk(const int32_t* p, int ex, int wt)
        : prefix(p), experts(ex), wtiles(wt), e(0), total((int64_t)p[ex] * wt)
    {
    }
    // item < total, not before the last one
    __device__ __forceinline__ void at(int64_t item, int& wtile, int& ttile)
    {
        // first expert whose tiles end behind item
        int lo = e, hi = experts - 1;
        if (item < (int64_t)prefix[lo + 1] * wtiles)
            hi = lo;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (item < (int64_t)prefix[mid + 1] * wtiles)
                hi = mid;
            else
                lo = mid + 1;
        }
        e = lo;
        const int tt = prefix[e + 1] - prefix[e];
        const int idx = (int)(item - (int64_t)prefix[e] * wtiles);
        wtile = idx / tt;
        ttile = idx - wtile * tt;
    }
};

// Tensor maps: weight codes, token codes, and for pairs the scale atoms of
// both (rows of 8-byte words; a CTA alone fetches them by plain bulk copies).
struct Maps {
    CUtensorMap w, a, ws, as;
};

template <bool PAIR, bool NV, bool F32>
__global__ void __launch_bounds__(GTHREADS, 1)
    expert_gemm_kernel(const __grid_constant__ Maps maps, ExpertGemmArgs p)
{
    using T = Tile<PAIR>;
    constexpr int TN = T::TN;
    extern __shared__ uint8_t raw_smem[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(raw_smem) + ALIGN_SLACK - 1) & ~uintptr_t(ALIGN_SLACK - 1));
    uint8_t* fixed = smem + T::STAGES * T::STAGE;
    const uint32_t smem_base = sptr(smem);
    const uint32_t bars = sptr(fixed);
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (T::STAGES + s); };
    auto acc_full = [&](int b) { return bars + 8 * (2 * T::STAGES + b); };
    auto acc_free = [&](int b) { return bars + 8 * (2 * T::STAGES + 2 + b); };
    int32_t* prefix = reinterpret_cast<int32_t*>(fixed + 256);
    volatile int* abort_flag = reinterpret_cast<int*>(fixed + 256 + (FP4Q_MAX_EXPERTS + 1) * 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fixed + 256 + (FP4Q_MAX_EXPERTS + 1) * 4 + 4);

    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;  // clusters are pairs of neighbours

    if (threadIdx.x == 0) {
        for (int s = 0; s < T::STAGES; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            bar_init(acc_full(b), 1);
            bar_init(acc_free(b), 4 * T::CTAS);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        __syncwarp();
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sptr(tmem_slot)),
                         "r"((uint32_t)T::COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sptr(tmem_slot)),
                         "r"((uint32_t)T::COLS)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    pdl_begin();
    // Token tiles of each expert, then of the experts before it; segments outside
    // the buffer count none, and all together no more than disjoint segments can have.
    for (int e = threadIdx.x; e < p.experts; e += GTHREADS) {
        const int64_t c = p.counts[e], s = p.starts[e];
        prefix[e + 1] = c > 0 && s >= 0 && s % kSegRows == 0 && s + c <= p.rows ? (int)((c + TN - 1) / TN) : 0;
    }
    if (threadIdx.x == 0)
        prefix[0] = 0;
    __syncthreads();
    if (warp == 0) {
        const int limit = (int)(p.rows / kSegRows);
        int carry = 0;
        for (int e0 = 0; e0 < p.experts; e0 += 32) {
            const int e = e0 + lane;
            int inc = e < p.experts ? prefix[e + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                inc += lane >= d ? v : 0;
            }
            inc = min(carry + inc, limit);
            if (e < p.experts)
                prefix[e + 1] = inc;
            carry = __shfl_sync(0xFFFFFFFFu, inc, 31);
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (PAIR)
        cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;

    const int wtiles = (p.N + WROWS - 1) / WROWS;            // of an expert
    const int wunits = (wtiles + T::CTAS - 1) / T::CTAS;     // tiles of a CTA or pair
    const int chunks = (p.K + CHUNK - 1) / CHUNK;
    constexpr int APC = NV ? 4 : 2;                              // scale atoms of a chunk
    const int atoms = NV ? (p.K + 63) / 64 : (p.K + 127) / 128;  // along a row
    const int64_t first_item = blockIdx.x / T::CTAS, step = gridDim.x / T::CTAS;
    Walk walk(prefix, p.experts, wunits);
    // columns of an MMA: a multiple of 16, of 32 for a pair (each half a multiple of 16)
    auto columns = [](int valid) { return PAIR ? (valid + 31) & ~31 : (valid + 15) & ~15; };

    if (warp == 0) {
        const bool leader = elect_one();
        const int lead = __ffs(__ballot_sync(0xFFFFFFFFu, leader)) - 1;
        int it = 0;
        bool ok = true;
        for (int64_t item = first_item; ok && item < walk.total; item += step) {
            int wt, tt;
            walk.at(item, wt, tt);
            wt = wt * T::CTAS + rank;
            const int row0 = p.starts[walk.e] + tt * TN;
            const int valid = min(TN, p.counts[walk.e] - tt * TN);
            const int wrow = walk.e * p.N + wt * WROWS;
            const int arow = row0 + rank * (columns(valid) / 2);
            const int boxes = PAIR ? 1 : (valid + T::BOX - 1) / T::BOX;
            const uint8_t* ws = p.w_scales + ((int64_t)walk.e * wtiles + wt) * atoms * ATOM;
            const uint8_t* as = p.a_scales + (int64_t)(row0 / 128) * atoms * ATOM;
            for (int c = 0; c < chunks; ++c, ++it) {
                const int s = it % T::STAGES;
                if (it >= T::STAGES && !bar_wait(empty(s), ((it / T::STAGES) & 1) ^ 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t st = smem_base + s * T::STAGE;
                const uint32_t sc = st + T::WBYTES + T::ABYTES;
                if (leader) {
                    if constexpr (PAIR) {
                        // both CTAs' bytes count on the first one's barrier
                        const uint32_t bar = in_first(full(s));
                        if (rank == 0)
                            bar_expect(full(s), 2 * (T::WBYTES + T::ABYTES + APC * ATOM * 3));
                        tma_box<true>(st, &maps.w, c * 128, wrow, bar);
                        tma_box<true>(st + T::WBYTES, &maps.a, c * 128, arow, bar);
                        tma_box<true>(sc, &maps.ws, c * APC * (ATOM / 8), walk.e * wtiles + wt, bar);
                        tma_box<true>(sc + T::SW, &maps.as, c * APC * (ATOM / 8), row0 / 128, bar);
                    } else {
                        const uint32_t n = ATOM * min(APC, atoms - c * APC);
                        bar_expect(full(s), T::WBYTES + boxes * T::BOX * 128 + 2 * n);
                        tma_box<false>(st, &maps.w, c * 128, wrow, full(s));
                        for (int b = 0; b < boxes; ++b)
                            tma_box<false>(st + T::WBYTES + b * T::BOX * 128, &maps.a, c * 128,
                                           arow + b * T::BOX, full(s));
                        bulk_load(sc, ws + (int64_t)c * APC * ATOM, n, full(s));
                        bulk_load(sc + T::SW, as + (int64_t)c * APC * ATOM, n, full(s));
                    }
                }
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        it = __shfl_sync(0xFFFFFFFFu, it, lead);  // stages issued
        // The releases of the last stages are arrivals of commits that nothing above waits for,
        // a pair's in both CTAs: they land before the memory of their barriers is given back.
        for (int j = it < T::STAGES ? 0 : it - T::STAGES; ok && j < it; ++j)
            ok = __all_sync(0xFFFFFFFFu, bar_wait(empty(j % T::STAGES), (j / T::STAGES) & 1, abort_flag));
        if (!ok) {
            if (lane == 0)
                atomicAdd(p.err, 1u);
            // copies in flight land before the CTA gives its memory back (a pair's
            // second CTA cannot see the barrier they count on: it waits as long)
            for (int j = it < T::STAGES ? 0 : it - T::STAGES; j < it; ++j)
                for (uint32_t i = 0; i < POLLS / 16 && !bar_poll(full(j % T::STAGES), (j / T::STAGES) & 1); ++i)
                    ;
        }
    } else if (warp == 1 && rank == 0) {
        const bool leader = elect_one();
        const int lead = __ffs(__ballot_sync(0xFFFFFFFFu, leader)) - 1;
        int it = 0, tile = 0;
        bool ok = true;
        for (int64_t item = first_item; ok && item < walk.total; item += step, ++tile) {
            int wt, tt;
            walk.at(item, wt, tt);
            const int valid = min(TN, p.counts[walk.e] - tt * TN);
            const int cols = __shfl_sync(0xFFFFFFFFu, columns(valid), 0);
            const int groups = TN == 128 ? 1 : (cols > 128 ? 2 : 1);
            const int buf = tile & 1;
            // buffers apart: tile - 2 has been read; overlapping: the shared
            // columns of tile - 1 have
            if (T::SHARE > 0 ? tile >= 1 : tile >= 2) {
                const int b = T::SHARE > 0 ? buf ^ 1 : buf;
                const int phase = T::SHARE > 0 ? (tile - 1) / 2 : (tile - 2) / 2;
                if (!__all_sync(0xFFFFFFFFu, bar_wait(acc_free(b), phase & 1, abort_flag))) {
                    ok = false;
                    break;
                }
            }
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + buf * T::SECOND;
            // instruction descriptor: E2M1 x E2M1, columns / 8 at bit 17, scale type (0 E4M3,
            // 1 E8M0) at bit 23, rows / 16 at bit 24; scale byte pair of MXFP4 at bits 4 and 29
            const uint32_t idesc = (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) |
                                   ((NV ? 0u : 1u) << 23) | ((WROWS * T::CTAS >> 4) << 24);
            for (int c = 0; c < chunks; ++c, ++it) {
                const int s = it % T::STAGES;
                if (!bar_wait(full(s), (it / T::STAGES) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t st = smem_base + s * T::STAGE;
                const uint32_t sc = st + T::WBYTES + T::ABYTES;
                const uint64_t da = desc_codes(st), db = desc_codes(st + T::WBYTES);
                const uint64_t dsw = desc_scales(sc), dsa = desc_scales(sc + T::SW);
                const int steps = min(CHUNK / 64, (p.K - c * CHUNK + 63) / 64);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < CHUNK / 64; ++k) {
                        if (k >= steps)
                            break;
                        const int a = NV ? k : k / 2;                // scale atom of this step
                        const uint32_t id = NV ? 0u : 2u * (k & 1);  // its byte pair
                        const uint32_t tsw = tmem + T::COL_SW + 4 * a;
                        const uint32_t tsa = tmem + T::COL_SA + 4 * (TN / 128) * a;
                        if (id == 0) {
                            copy_scales<PAIR>(tsw, dsw + a * (ATOM >> 4));
                            copy_scales<PAIR>(tsa, dsa + a * (ATOM >> 4));
                            if (TN > 128 && groups > 1)
                                copy_scales<PAIR>(tsa + 4, dsa + (APC + a) * (ATOM >> 4));
                        }
                        mma<PAIR, NV>(d, da + 2 * k, db + 2 * k, idesc | (id << 4) | (id << 29), tsw, tsa,
                                (c | k) != 0);
                    }
                    commit<PAIR>(empty(s));
                }
            }
            if (ok && leader)
                commit<PAIR>(acc_full(buf));
            ok = __all_sync(0xFFFFFFFFu, ok);
        }
        if (!ok) {
            if (lane == 0)
                atomicAdd(p.err, 1u);
            // products in flight end before their memory is given back
            const int j = __shfl_sync(0xFFFFFFFFu, it, lead) - 1;
            for (uint32_t i = 0; j >= 0 && i < POLLS / 16 &&
                                 !bar_poll(empty(j % T::STAGES), (j / T::STAGES) & 1); ++i)
                ;
        }
    } else if (warp >= 2) {
        const int quarter = warp & 3;  // TMEM lanes 32 quarter .. + 31
        int tile = 0;
        bool ok = true;
        for (int64_t item = first_item; ok && item < walk.total; item += step, ++tile) {
            int wt, tt;
            walk.at(item, wt, tt);
            wt = wt * T::CTAS + rank;
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
            const int m0 = wt * WROWS + 32 * quarter;  // this warp's outputs m0 .. m0 + 31
            const int nm = p.N - m0;                   // of which nm exist
            const int64_t at = (int64_t)row0 * p.N + m0;
            auto release = [&]() {
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR)
                        bar_arrive_first(in_first(acc_free(buf)));
                    else
                        bar_arrive(acc_free(buf));
                }
            };
            // columns col .. col + 15 (rows of d): read, scaled, stored
            auto part = [&](int col, bool last) {
                uint32_t v[16];
                tmem_load16(acc + col, v);
                if (last)
                    release();
                const int n = valid - col;  // columns that are rows of d
                if constexpr (F32) {
                    float* out = static_cast<float*>(p.d) + at + (int64_t)col * p.N + lane;
                    if (lane < nm) {
#pragma unroll
                        for (int i = 0; i < 16; ++i, out += p.N)
                            if (i < n)
                                *out = __fmul_rn(__uint_as_float(v[i]), alpha);
                    }
                } else {
                    // Neighbouring lanes swap one of two columns, so that a lane
                    // holds two neighbouring outputs of one row: one 4-byte store for two
                    // columns, 64 contiguous bytes a row.
                    const bool odd = lane & 1;
                    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.d) + at +
                                         (int64_t)(col + odd) * p.N + (lane & ~1);
                    const bool mine = (lane & ~1) < nm;
#pragma unroll
                    for (int i = 0; i < 16; i += 2, out += 2 * (int64_t)p.N) {
                        const float a = __fmul_rn(__uint_as_float(v[i]), alpha);
                        const float b = __fmul_rn(__uint_as_float(v[i + 1]), alpha);
                        const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1);
                        const uint32_t w = odd ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
                        if (mine && i + (int)odd < n)
                            *reinterpret_cast<uint32_t*>(out) = w;
                    }
                }
            };
            if constexpr (T::SHARE > 0) {
                // the columns that the other buffer shares come first
                const int first = buf == 0 ? TN - T::SHARE : 0;
                for (int col = first; col < first + T::SHARE; col += 16)
                    part(col, col + 16 == first + T::SHARE);
                const int lo = buf == 0 ? 0 : T::SHARE;
                for (int col = lo; col < lo + TN - T::SHARE && col < valid; col += 16)
                    part(col, false);
            } else {
                for (int col = 0; col < valid; col += 16)
                    part(col, col + 16 >= valid);
            }
        }
        if (!ok && lane == 0)
            atomicAdd(p.err, 1u);
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (PAIR)  // neither leaves while the other's MMAs or arrivals may reach it
        cluster_sync();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if constexpr (PAIR)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)T::COLS));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)T::COLS));
    }
}

template <bool PAIR, bool NV, bool F32>
cudaError_t gemm_one(const uint8_t* a_codes, const uint8_t* w_codes, const ExpertGemmArgs& a, int dev,
                     int sms, cudaStream_t st)
{
    using T = Tile<PAIR>;
    Maps maps = {};
    bool ok = make_byte_map(&maps.w, w_codes, a.K / 2, (int64_t)a.experts * a.N, WROWS) &&
              make_byte_map(&maps.a, a_codes, a.K / 2, a.rows, T::BOX);
    if (PAIR) {
        const int64_t words = (NV ? (a.K + 63) / 64 : (a.K + 127) / 128) * (ATOM / 8);  // of a row of atoms
        const int box = (NV ? 4 : 2) * (ATOM / 8);
        ok = ok && make_word_map(&maps.ws, a.w_scales, words, (int64_t)a.experts * ((a.N + 127) / 128), box, 1) &&
             make_word_map(&maps.as, a.a_scales, words, a.rows / 128, box, T::TN / 128);
    }
    if (!ok)
        return cudaErrorInvalidValue;
    auto kern = expert_gemm_kernel<PAIR, NV, F32>;
    static std::atomic<uint64_t> done{0};
    if (cudaError_t e = allow_smem(kern, T::SMEM, dev, done))
        return e;
    if (!PAIR)
        return launch_pdl(kern, dim3((unsigned)sms), dim3(GTHREADS), T::SMEM, st, maps, a);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(sms & ~1));
    cfg.blockDim = dim3(GTHREADS);
    cfg.dynamicSmemBytes = T::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

template <bool PAIR>
cudaError_t gemm_type(bool nv, bool out32, const uint8_t* a_codes, const uint8_t* w_codes,
                      const ExpertGemmArgs& a, int dev, int sms, cudaStream_t st)
{
    if (nv)
        return out32 ? gemm_one<PAIR, true, true>(a_codes, w_codes, a, dev, sms, st)
                     : gemm_one<PAIR, true, false>(a_codes, w_codes, a, dev, sms, st);
    return out32 ? gemm_one<PAIR, false, true>(a_codes, w_codes, a, dev, sms, st)
                 : gemm_one<PAIR, false, false>(a_codes, w_codes, a, dev, sms, st);
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
    if (mean_rows <= 128)
        return gemm_type<false>(nv, out32, a_codes, w_codes, a, dev, sms, st);
    return gemm_type<true>(nv, out32, a_codes, w_codes, a, dev, sms, st);
}

}  // namespace fp4q

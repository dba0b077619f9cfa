// expert_sort.cu -- stable counting sort of the router's choices by expert.
//
//   counts[e] = #{i : ids[i] = e},  starts[e] = sum_{f < e} 128 ceil(counts[f] / 128),
//   slots[i]  = starts[e] + #{i' < i : ids[i'] = e}  for e = ids[i], -1 if e is no expert.
//
// A block of up to 32 warps takes SUB choices at a time, held in registers
// (one contiguous run of 32-wide steps per warp). __match_any_sync gives a
// choice its rank among the equal ids of its step, a per-warp counter in
// shared memory its rank within the warp's run, an exclusive scan of those
// counters over the warps its rank within the block. Ranks are positions, so no
// atomic's order enters the result.
//
// Up to SUB choices one block does it all in one launch: what counts is
// the launch and a dozen barriers, not bandwidth. Above, a first kernel counts the ids of each
// block's chunk (one block per SM at most), and the second adds up the counts of the blocks
// before it; it reads the ids a second time, from L2. (64 x 2 choices of 8 experts: a kernel of 5 us;
// 65536 x 8 of 256: 4 and 15 us, 19.5 cold with the launches, of which reading 4 MB would take 1.)
#include "experts.h"
#include "fp4q_device.cuh"

namespace fp4q {

namespace {

constexpr int STEPS = 4;               // 32-wide steps per warp, ids in registers
constexpr int MAXW = 32;               // warps of a block
constexpr int SUB = MAXW * 32 * STEPS; // 4096 choices per pass of a block
constexpr int MAX_BLOCKS = 148;

template <class Id>
__device__ __forceinline__ int expert_of(const Id* ids, int64_t i, int64_t end, int experts)
{
    if (i >= end)
        return -1;
    const Id v = ids[i];
    return v >= 0 && v < (Id)experts ? (int)v : -1;
}

template <class Id>
__global__ void __launch_bounds__(1024) sort_count_kernel(SortArgs a)
{
    extern __shared__ int32_t hist[];
    pdl_begin();
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
        hist[e] = 0;
    __syncthreads();
    const int64_t lo = blockIdx.x * a.chunk, hi = min(a.n, lo + a.chunk);
    for (int64_t i0 = lo + threadIdx.x; i0 < hi; i0 += STEPS * blockDim.x) {
        int e[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            e[s] = expert_of(static_cast<const Id*>(a.ids), i0 + s * blockDim.x, hi, a.experts);
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            if (e[s] >= 0)
                atomicAdd(&hist[e[s]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x)
        a.hist[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

// Shared memory: rank counters [warps][experts], then per expert base (the next free
// row for this block), its padded size and this pass's count.
template <class Id>
__global__ void __launch_bounds__(1024) sort_place_kernel(SortArgs a)
{
    extern __shared__ int32_t sm[];
    const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int E = a.experts;
    int32_t* cnt = sm;
    int32_t* base = sm + warps * E;
    __shared__ int32_t carry_sm;
    pdl_begin();
    const int64_t lo = blockIdx.x * a.chunk, hi = min(a.n, lo + a.chunk);
    const bool alone = gridDim.x == 1;
    const int per_warp = (int)((min((int64_t)SUB, a.chunk) + blockDim.x - 1) / blockDim.x);  // steps

    for (int64_t sub = lo; sub < hi || sub == lo; sub += SUB) {
        const bool first = sub == lo;
        int e[STEPS], rank[STEPS];
        const int64_t run = sub + (int64_t)warp * per_warp * 32;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
            e[s] = s < per_warp ? expert_of(static_cast<const Id*>(a.ids), run + 32 * s + lane, hi, E) : -1;
        for (int i = threadIdx.x; i < (first ? warps + 2 : warps) * E; i += blockDim.x)
            cnt[i] = 0;  // and base behind them
        __syncthreads();
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            if (s < per_warp) {  // uniform
                const unsigned same = __match_any_sync(0xFFFFFFFFu, e[s]);
                const int before = __popc(same & ((1u << lane) - 1));
                int old = 0;
                if (e[s] >= 0)
                    old = cnt[warp * E + e[s]];
                __syncwarp();
                if (e[s] >= 0 && before == 0)
                    cnt[warp * E + e[s]] = old + __popc(same);
                __syncwarp();
                rank[s] = old + before;
            }
        }
        __syncthreads();
        // The counts of the blocks before this one and of all, once: a thread
        // adds up every parts-th block of an expert, shared memory the parts
        // (sums of whole numbers: the order does not matter).
        if (first && !alone) {
            const int parts = max(1, (int)blockDim.x / E);
            for (int x = threadIdx.x; x < parts * E; x += blockDim.x) {
                const int e1 = x % E;
                int before = 0, total = 0;
#pragma unroll 8
                for (int b = x / E; b < (int)gridDim.x; b += parts) {
                    const int c = a.hist[(int64_t)b * E + e1];
                    before += b < (int)blockIdx.x ? c : 0;
                    total += c;
                }
                atomicAdd(&base[e1], before);
                atomicAdd(&base[E + e1], total);
            }
            __syncthreads();
        }
        // counters -> exclusive over the warps
        for (int x = threadIdx.x; x < E; x += blockDim.x) {
            int sum = 0;
            for (int w = 0; w < warps; ++w) {
                const int c = cnt[w * E + x];
                cnt[w * E + x] = sum;
                sum += c;
            }
            if (first) {
                const int total = alone ? sum : base[E + x];
                if (blockIdx.x == 0)
                    a.counts[x] = total;
                // the padded size, for the scan over experts
                base[E + x] = (total + kSegRows - 1) / kSegRows * kSegRows;
            }
            base[2 * E + x] = sum;  // this pass's total
        }
        __syncthreads();
        if (first) {
            if (warp == 0) {
                int carry = 0;
                for (int x0 = 0; x0 < E; x0 += 32) {
                    const int x = x0 + lane;
                    const int v = x < E ? base[E + x] : 0;
                    int inc = v;
#pragma unroll
                    for (int d = 1; d < 32; d *= 2) {
                        const int t = __shfl_up_sync(0xFFFFFFFFu, inc, d);
                        inc += lane >= d ? t : 0;
                    }
                    if (x < E) {
                        const int start = carry + inc - v;
                        base[x] += start;
                        if (blockIdx.x == 0)
                            a.starts[x] = start;
                    }
                    carry += __shfl_sync(0xFFFFFFFFu, inc, 31);
                }
                if (lane == 0)
                    carry_sm = carry;
            }
            __syncthreads();
            if (threadIdx.x == 0 && blockIdx.x == 0)
                a.starts[E] = carry_sm;
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int64_t i = run + 32 * s + lane;
            if (s < per_warp && i < hi)
                a.slots[i] = e[s] >= 0 ? base[e[s]] + cnt[warp * E + e[s]] + rank[s] : -1;
        }
        __syncthreads();
        for (int x = threadIdx.x; x < E; x += blockDim.x)
            base[x] += base[2 * E + x];
    }
}

// Dynamic shared memory of the placing kernel.
size_t place_smem(int warps, int experts)
{
    return ((size_t)warps + 3) * experts * sizeof(int32_t);
}

template <class Id>
cudaError_t sort_impl(const SortArgs& a, cudaStream_t st)
{
    const int64_t blocks = sort_blocks(a.n);
    SortArgs b = a;
    int threads = 1024;
    if (blocks == 1) {
        // one step per warp while there are warps to take it
        const int64_t warps = (a.n + 31) / 32;
        threads = 32 * (int)(warps < 4 ? 4 : (warps < MAXW ? warps : MAXW));
        b.chunk = SUB;
        if (a.n < threads)
            b.chunk = threads;
        else if (a.n <= SUB)
            b.chunk = a.n;
    } else {
        b.chunk = ((a.n + blocks - 1) / blocks + 1023) / 1024 * 1024;
        cudaError_t e = launch_pdl(sort_count_kernel<Id>, dim3((unsigned)blocks), dim3(1024),
                                   a.experts * sizeof(int32_t), st, b);
        if (e != cudaSuccess)
            return e;
    }
    const size_t smem = place_smem(threads / 32, a.experts);
    // The limit belongs to the kernel, not to a call: the most that any call needs, once per
    // device, so that no call depends on the sizes of others (before this one, or on other threads).
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess)
        e = allow_smem(sort_place_kernel<Id>, place_smem(MAXW, FP4Q_MAX_EXPERTS), dev, done);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(sort_place_kernel<Id>, dim3((unsigned)blocks), dim3(threads), smem, st, b);
}

}  // namespace

// Blocks of a sort: one up to SUB choices, then one per SUB, at most one per SM
// of the device the library is built for.
int64_t sort_blocks(int64_t n)
{
    const int64_t b = (n + SUB - 1) / SUB;
    return b < 1 ? 1 : (b > MAX_BLOCKS ? MAX_BLOCKS : b);
}

cudaError_t launch_expert_sort(const SortArgs& a, int id_bytes, cudaStream_t st)
{
    return id_bytes == 8 ? sort_impl<int64_t>(a, st) : sort_impl<int32_t>(a, st);
}

}  // namespace fp4q

// experts.h -- argument blocks and launchers of the mixture-of-experts entry
// points (experts_api.cu and the expert_*.cu kernels).
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime_api.h>

#include "fp4q_experts.h"
#include "internal.h"

namespace fp4q {

// Host helpers defined in api.cu: the per-device error counter's address, and
// cuTensorMapEncodeTiled for a row-major matrix of bytes (128-byte swizzle, a
// box of 128 bytes x box_rows rows); false if the driver refuses it.
cudaError_t device_error_word(unsigned** p);
bool make_byte_map(CUtensorMap* map, const void* base, int64_t row_bytes, int64_t rows, int box_rows);
// The same for a matrix of 8-byte words without swizzle, a box of box_words x box_rows.
bool make_word_map(CUtensorMap* map, const void* base, int64_t row_words, int64_t rows, int box_words,
                   int box_rows);

// Raises a kernel's dynamic shared memory limit, once per kernel (`done`, a
// bit per device ordinal below 64) and device.
template <class K>
cudaError_t allow_smem(K kernel, size_t bytes, int dev, std::atomic<uint64_t>& done)
{
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (bit != 0 && (done.load(std::memory_order_acquire) & bit))
        return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_release);
    return e;
}

constexpr int kSegRows = 128;  // every expert's segment starts at a multiple of this

struct SortArgs {
    const void* ids;
    int64_t n;
    int experts;
    int32_t* counts;
    int32_t* starts;
    int32_t* slots;
    int32_t* hist;      // [blocks][experts] per-block counts (several blocks only)
    int64_t chunk;      // choices of one block
};
int64_t sort_blocks(int64_t n);
cudaError_t launch_expert_sort(const SortArgs& a, int id_bytes, cudaStream_t st);

// Segments of a row quantizer's call: room for a few grid steps below 2^32.
constexpr int64_t kMaxSegs = 0xF0000000ll;

// Rows quantized into the MMA layout, from tokens (k destinations each) or
// from the gated activation of rows (one destination).
struct RowQuantArgs {
    const uint16_t* x;      // bf16 tokens [n, cols], or gate and value [rows, 2 cols]
    uint32_t n;             // tokens, or rows taken
    uint32_t nseg;          // 32-element segments: n * spr, at most kMaxSegs
    uint32_t spr;           // segments per row = cols / 32
    uint32_t atoms_k;       // 4-block atoms per 128 rows along a row
    const int32_t* slots;   // [n, k] destination rows; NULL: row i itself (glu only)
    int k;
    int64_t rows;           // rows of the outputs; slots outside are skipped
    int act;                // glu: fp4q_activation
    const float* amax;      // NVFP4: device abs-max, or the parts' maxima
    int amax_parts;         // 0: *amax is the abs-max; else their number
    float* sg_out;
    uint8_t* codes;
    uint8_t* scales;
    void* dq;
    int dq_kind;            // 0 none, 1 fp32, 2 bf16
    uint32_t keep;          // 0xFFFFFFFF, passed at run time (see encode_seg)
    float* amax_out;        // abs-max pass: one maximum of each CTA
};
// strat: KStrat of NVFP4 (block 16) or MXFP4 (block 32).
cudaError_t launch_token_quant(int strat, int rot, const RowQuantArgs& a, cudaStream_t st);
cudaError_t launch_glu_quant_nv(int strat, int rot, const RowQuantArgs& a, cudaStream_t st);
cudaError_t launch_glu_quant_mx(int strat, int rot, const RowQuantArgs& a, cudaStream_t st);
// The abs-max pass: maxima of the rotated tokens, or of the rotated gated
// activation, into a.amax_out; their number (at most FP4Q_AMAX_WORK) into *parts.
cudaError_t launch_token_amax(int rot, const RowQuantArgs& a, int* parts, cudaStream_t st);
cudaError_t launch_glu_amax(int rot, const RowQuantArgs& a, int* parts, cudaStream_t st);

struct GluBwdArgs {
    const uint16_t* gu;
    const uint16_t* dh;
    uint16_t* dgu;
    const int32_t* slots;
    int64_t n;              // rows taken
    int64_t rows;
    int64_t cols;
    int act;
};
cudaError_t launch_glu_bwd(int rot, const GluBwdArgs& a, cudaStream_t st);

struct CombineArgs {
    const void* y;
    int64_t rows, cols;
    const int32_t* slots;
    int64_t tokens;
    int k;
    const float* weights;
    void* out;
};
cudaError_t launch_combine(bool y32, bool out32, int rot, const CombineArgs& a, cudaStream_t st);

struct CombineBwdArgs {
    const void* g;
    const void* y;
    int64_t rows, cols;
    const int32_t* slots;
    int64_t tokens;
    int k;
    const float* weights;
    void* dy;
    float* dw;
};
cudaError_t launch_combine_bwd(bool g32, bool y32, const CombineBwdArgs& a, cudaStream_t st);

struct ExpertGemmArgs {
    const uint8_t* w_scales;
    const uint8_t* a_scales;
    const float* a_sg;      // NVFP4 s_g of the rows, else NULL
    const float* w_sg;      // NVFP4 s_g of each expert, else NULL
    const int32_t* counts;
    const int32_t* starts;
    void* d;
    unsigned* err;          // device error counter
    int64_t rows;
    int experts;
    int N, K;
};
cudaError_t launch_expert_gemm(bool nv, bool out32, int64_t mean_rows, const uint8_t* a_codes,
                               const uint8_t* w_codes, const ExpertGemmArgs& a, cudaStream_t st);

}  // namespace fp4q

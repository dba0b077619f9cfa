// experts_api.cu -- the extern "C" entry points of include/fp4q_experts.h.
//
// Host side only: validate every argument, then enqueue kernels on the
// caller's stream. Nothing is allocated and nothing is synchronised.
#include <cstdint>

#include "experts.h"

using namespace fp4q;

namespace {

constexpr int64_t kMaxRows = 0x7FFFFFFF;       // padded rows fit an int32
constexpr int64_t kMaxElems = (int64_t)1 << 40;

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
bool valid_rot(int rot) { return rot == 0 || rot == 16 || rot == 32 || rot == 64 || rot == 128; }
bool valid_dtype(int t) { return t == FP4Q_OUT_F32 || t == FP4Q_OUT_BF16; }
bool valid_act(int a) { return a == FP4Q_ACT_SILU || a == FP4Q_ACT_GELU_TANH; }

// rows x cols elements within limits
bool valid_size(int64_t rows, int64_t cols)
{
    return rows >= 0 && cols >= 0 && rows <= kMaxRows && (cols == 0 || rows <= kMaxElems / cols);
}

// The quantizer's arguments shared by fp4q_expert_quantize and
// fp4q_glu_quantize, without the shape of the input.
fp4q_status check_quant(int64_t rows, int64_t cols, int fmt, int strat, int rot,
                        const float* amax_in, const float* sg_out, const float* amax_work,
                        const void* dq, int dq_dtype)
{
    if (fmt != FP4Q_FMT_NVFP4 && fmt != FP4Q_FMT_MXFP4)
        return FP4Q_ERR_UNSUPPORTED;
    if (strat < FP4Q_ABSMAX || strat > FP4Q_BRUTE_FORCE)
        return FP4Q_ERR_UNSUPPORTED;
    if (fmt == FP4Q_FMT_MXFP4 && strat != FP4Q_ABSMAX && strat != FP4Q_BRUTE_FORCE)
        return FP4Q_ERR_UNSUPPORTED;
    if (!valid_rot(rot) || (dq != nullptr && !valid_dtype(dq_dtype)))
        return FP4Q_ERR_UNSUPPORTED;
    if (!valid_size(rows, cols) || cols % 32 != 0 || (rot > 0 && cols % rot != 0))
        return FP4Q_ERR_SHAPE;
    if (fmt == FP4Q_FMT_NVFP4) {
        if (sg_out == nullptr || (amax_in == nullptr && amax_work == nullptr))
            return FP4Q_ERR_NULL;
        if (misaligned(sg_out, 4) || misaligned(amax_in, 4) || misaligned(amax_work, 4))
            return FP4Q_ERR_ALIGN;
        if (amax_in == sg_out || (amax_in == nullptr && amax_work == sg_out))
            return FP4Q_ERR_ALIAS;
    }
    return FP4Q_OK;
}

int strat_id(int fmt, int strat)
{
    return fmt == FP4Q_FMT_NVFP4 ? strat : (strat == FP4Q_BRUTE_FORCE ? K_MX_BRUTE : K_MX);
}

RowQuantArgs row_args(const void* x, int64_t count, int64_t rows, int64_t cols, int k,
                      const int32_t* slots, int act, int fmt, float* sg_out, uint8_t* codes,
                      uint8_t* scales, void* dq, int dq_dtype)
{
    RowQuantArgs a;
    a.x = static_cast<const uint16_t*>(x);
    a.spr = (uint32_t)(cols / 32);
    a.n = (uint32_t)count;
    a.nseg = (uint32_t)(count * (cols / 32));
    const int block = fmt == FP4Q_FMT_NVFP4 ? 16 : 32;
    a.atoms_k = (uint32_t)((cols / block + 3) / 4);
    a.slots = slots;
    a.k = k;
    a.rows = rows;
    a.act = act;
    a.amax = nullptr;
    a.amax_parts = 0;
    a.sg_out = fmt == FP4Q_FMT_NVFP4 ? sg_out : nullptr;
    a.codes = codes;
    a.scales = scales;
    a.dq = dq;
    a.dq_kind = dq == nullptr ? 0 : (dq_dtype == FP4Q_OUT_F32 ? 1 : 2);
    a.keep = 0xFFFFFFFFu;
    a.amax_out = nullptr;
    return a;
}

}  // namespace

extern "C" {

int64_t fp4q_expert_rows(int64_t n, int64_t experts)
{
    if (n < 0 || n > kMaxRows || experts < 1 || experts > FP4Q_MAX_EXPERTS)
        return -1;
    const int64_t used = n < experts ? n : experts;
    const int64_t rows = (n + (kSegRows - 1) * used) / kSegRows * kSegRows;
    return rows <= kMaxRows ? rows : -1;
}

int64_t fp4q_expert_sort_work(int64_t n, int64_t experts)
{
    if (fp4q_expert_rows(n, experts) < 0)
        return -1;
    const int64_t blocks = sort_blocks(n);
    return blocks == 1 ? 0 : blocks * experts * (int64_t)sizeof(int32_t);
}

fp4q_status fp4q_expert_sort(const void* ids, int id_bytes, int64_t n, int64_t experts,
                             int32_t* counts, int32_t* starts, int32_t* slots, void* work,
                             cudaStream_t stream)
{
    if (id_bytes != 4 && id_bytes != 8)
        return FP4Q_ERR_UNSUPPORTED;
    const int64_t need = fp4q_expert_sort_work(n, experts);
    if (need < 0)
        return FP4Q_ERR_SHAPE;
    if (counts == nullptr || starts == nullptr || (n > 0 && (ids == nullptr || slots == nullptr)) ||
        (need > 0 && work == nullptr))
        return FP4Q_ERR_NULL;
    if (misaligned(ids, (uintptr_t)id_bytes) || misaligned(counts, 4) || misaligned(starts, 4) ||
        misaligned(slots, 4) || misaligned(work, 4))
        return FP4Q_ERR_ALIGN;
    if (cudaError_t ie = injected_launch_error())
        return record_cuda_error(ie);
    SortArgs a;
    a.ids = ids;
    a.n = n;
    a.experts = (int)experts;
    a.counts = counts;
    a.starts = starts;
    a.slots = slots;
    a.hist = static_cast<int32_t*>(work);
    a.chunk = 0;
    return record_cuda_error(launch_expert_sort(a, id_bytes, stream));
}

fp4q_status fp4q_expert_quantize(const void* x, int64_t tokens, int64_t cols, int k,
                                 const int32_t* slots, int64_t rows, fp4q_format fmt,
                                 fp4q_strategy strat, int rot, const float* global_amax_in,
                                 float* global_scale_out, float* amax_work, uint8_t* codes,
                                 uint8_t* mma_scales, void* dq, fp4q_dtype dq_dtype,
                                 cudaStream_t stream)
{
    fp4q_status st = check_quant(rows, cols, fmt, strat, rot, global_amax_in, global_scale_out,
                                 amax_work, dq, dq_dtype);
    if (st != FP4Q_OK)
        return st;
    if (k < 1 || k > FP4Q_MAX_CHOICES || rows % kSegRows != 0 || !valid_size(tokens, cols) ||
        tokens * (cols / 32) > kMaxSegs)
        return FP4Q_ERR_SHAPE;
    const int64_t n = tokens * cols;
    if (n > 0 && (x == nullptr || slots == nullptr))
        return FP4Q_ERR_NULL;
    if (n > 0 && rows > 0 && (codes == nullptr || mma_scales == nullptr))
        return FP4Q_ERR_NULL;
    if (misaligned(x, 16) || misaligned(slots, 4) || misaligned(codes, 16) ||
        misaligned(mma_scales, 16) || misaligned(dq, 16))
        return FP4Q_ERR_ALIGN;
    if (cudaError_t ie = injected_launch_error())
        return record_cuda_error(ie);
    const bool nv = fmt == FP4Q_FMT_NVFP4;
    if (n == 0)
        return nv ? record_cuda_error(launch_set_one(global_scale_out, stream)) : FP4Q_OK;
    RowQuantArgs a = row_args(x, tokens, rows, cols, k, slots, 0, fmt, global_scale_out, codes,
                              mma_scales, dq, dq_dtype);
    if (nv) {
        a.amax = global_amax_in;
        if (global_amax_in == nullptr) {
            a.amax_out = amax_work;
            if (cudaError_t e = launch_token_amax(rot, a, &a.amax_parts, stream))
                return record_cuda_error(e);
            a.amax = amax_work;
        }
    }
    return record_cuda_error(launch_token_quant(strat_id(fmt, strat), rot, a, stream));
}

fp4q_status fp4q_expert_gemm(const uint8_t* a_codes, const uint8_t* a_mma_scales,
                             const float* a_global_scale, const uint8_t* w_codes,
                             const uint8_t* w_mma_scales, const float* w_global_scale,
                             const int32_t* counts, const int32_t* starts, int64_t experts,
                             int64_t rows, int64_t N, int64_t K, fp4q_format fmt,
                             int64_t mean_rows, void* d, fp4q_dtype d_dtype, cudaStream_t stream)
{
    if (fmt != FP4Q_FMT_NVFP4 && fmt != FP4Q_FMT_MXFP4)
        return FP4Q_ERR_UNSUPPORTED;
    if (!valid_dtype(d_dtype))
        return FP4Q_ERR_UNSUPPORTED;
    const bool nv = fmt == FP4Q_FMT_NVFP4;
    const bool out32 = d_dtype == FP4Q_OUT_F32;
    if (experts < 1 || experts > FP4Q_MAX_EXPERTS || rows < 0 || rows > kMaxRows ||
        rows % kSegRows != 0 || N <= 0 || K <= 0 || K % 32 != 0 || N % (out32 ? 4 : 8) != 0 ||
        K > kMaxRows || N > kMaxRows || experts * N > kMaxRows - 1024 || mean_rows < 0)
        return FP4Q_ERR_SHAPE;
    if (rows == 0)
        return FP4Q_OK;
    if (a_codes == nullptr || a_mma_scales == nullptr || w_codes == nullptr ||
        w_mma_scales == nullptr || counts == nullptr || starts == nullptr || d == nullptr ||
        (nv && (a_global_scale == nullptr || w_global_scale == nullptr)))
        return FP4Q_ERR_NULL;
    if (misaligned(a_codes, 16) || misaligned(a_mma_scales, 16) || misaligned(w_codes, 16) ||
        misaligned(w_mma_scales, 16) || misaligned(d, 16) || misaligned(counts, 4) ||
        misaligned(starts, 4) ||
        (nv && (misaligned(a_global_scale, 4) || misaligned(w_global_scale, 4))))
        return FP4Q_ERR_ALIGN;
    if (cudaError_t ie = injected_launch_error())
        return record_cuda_error(ie);
    ExpertGemmArgs a;
    if (cudaError_t e = device_error_word(&a.err))
        return record_cuda_error(e);
    a.w_scales = w_mma_scales;
    a.a_scales = a_mma_scales;
    a.a_sg = nv ? a_global_scale : nullptr;
    a.w_sg = nv ? w_global_scale : nullptr;
    a.counts = counts;
    a.starts = starts;
    a.d = d;
    a.rows = rows;
    a.experts = (int)experts;
    a.N = (int)N;
    a.K = (int)K;
    return record_cuda_error(launch_expert_gemm(nv, out32, mean_rows, a_codes, w_codes, a, stream));
}

fp4q_status fp4q_glu_quantize(const void* gu, int64_t rows, int64_t cols, const int32_t* slots,
                              int64_t n, fp4q_activation act, fp4q_format fmt, fp4q_strategy strat,
                              int rot, const float* global_amax_in, float* global_scale_out,
                              float* amax_work, uint8_t* codes, uint8_t* mma_scales, void* dq,
                              fp4q_dtype dq_dtype, cudaStream_t stream)
{
    if (!valid_act(act))
        return FP4Q_ERR_UNSUPPORTED;
    fp4q_status st = check_quant(rows, cols, fmt, strat, rot, global_amax_in, global_scale_out,
                                 amax_work, dq, dq_dtype);
    if (st != FP4Q_OK)
        return st;
    const int64_t taken = slots == nullptr ? rows : n;
    if (!valid_size(rows, 2 * cols) || !valid_size(taken, cols) || taken * (cols / 32) > kMaxSegs)
        return FP4Q_ERR_SHAPE;
    const bool empty = taken == 0 || rows == 0 || cols == 0;
    if (!empty && (gu == nullptr || codes == nullptr || mma_scales == nullptr))
        return FP4Q_ERR_NULL;
    if (misaligned(gu, 16) || misaligned(slots, 4) || misaligned(codes, 16) ||
        misaligned(mma_scales, 16) || misaligned(dq, 16))
        return FP4Q_ERR_ALIGN;
    if (cudaError_t ie = injected_launch_error())
        return record_cuda_error(ie);
    const bool nv = fmt == FP4Q_FMT_NVFP4;
    if (empty)
        return nv ? record_cuda_error(launch_set_one(global_scale_out, stream)) : FP4Q_OK;
    RowQuantArgs a = row_args(gu, taken, rows, cols, 1, slots, act, fmt, global_scale_out, codes,
                              mma_scales, dq, dq_dtype);
    if (!nv)
        return record_cuda_error(launch_glu_quant_mx(strat_id(fmt, strat), rot, a, stream));
    a.amax = global_amax_in;
    if (global_amax_in == nullptr) {
        a.amax_out = amax_work;
        if (cudaError_t e = launch_glu_amax(rot, a, &a.amax_parts, stream))
            return record_cuda_error(e);
        a.amax = amax_work;
    }
    return record_cuda_error(launch_glu_quant_nv(strat, rot, a, stream));
}

fp4q_status fp4q_glu_bwd(const void* gu, const void* dh, int64_t rows, int64_t cols,
                         const int32_t* slots, int64_t n, fp4q_activation act, int rot, void* dgu,
                         cudaStream_t stream)
{
    if (!valid_act(act) || !valid_rot(rot))
        return FP4Q_ERR_UNSUPPORTED;
    const int64_t taken = slots == nullptr ? rows : n;
    if (!valid_size(rows, cols) || !valid_size(rows, 2 * cols) || !valid_size(taken, cols) ||
        cols % 8 != 0 || (rot > 0 && (cols % rot != 0 || cols % 32 != 0)))
        return FP4Q_ERR_SHAPE;
    if (taken == 0 || rows == 0 || cols == 0)
        return FP4Q_OK;
    if (gu == nullptr || dh == nullptr || dgu == nullptr)
        return FP4Q_ERR_NULL;
    if (misaligned(gu, 16) || misaligned(dh, 16) || misaligned(dgu, 16) || misaligned(slots, 4))
        return FP4Q_ERR_ALIGN;
    if (cudaError_t ie = injected_launch_error())
        return record_cuda_error(ie);
    GluBwdArgs a;
    a.gu = static_cast<const uint16_t*>(gu);
    a.dh = static_cast<const uint16_t*>(dh);
    a.dgu = static_cast<uint16_t*>(dgu);
    a.slots = slots;
    a.n = taken;
    a.rows = rows;
    a.cols = cols;
    a.act = act;
    return record_cuda_error(launch_glu_bwd(rot, a, stream));
}

fp4q_status fp4q_expert_combine(const void* y, fp4q_dtype y_dtype, int64_t rows, int64_t cols,
                                const int32_t* slots, int64_t tokens, int k, const float* weights,
                                int rot, void* out, fp4q_dtype out_dtype, cudaStream_t stream)
{
    if (!valid_dtype(y_dtype) || !valid_dtype(out_dtype) || !valid_rot(rot))
        return FP4Q_ERR_UNSUPPORTED;
    if (k < 1 || k > FP4Q_MAX_CHOICES || !valid_size(rows, cols) || !valid_size(tokens, cols) ||
        cols % 8 != 0 || (rot > 0 && cols % rot != 0))
        return FP4Q_ERR_SHAPE;
    if (tokens == 0 || cols == 0)
        return FP4Q_OK;
    if ((rows > 0 && y == nullptr) || slots == nullptr || out == nullptr)
        return FP4Q_ERR_NULL;
    if (misaligned(y, 16) || misaligned(slots, 4) || misaligned(weights, 4) || misaligned(out, 16))
        return FP4Q_ERR_ALIGN;
    if (cudaError_t ie = injected_launch_error())
        return record_cuda_error(ie);
    CombineArgs a;
    a.y = y;
    a.rows = rows;
    a.cols = cols;
    a.slots = slots;
    a.tokens = tokens;
    a.k = k;
    a.weights = weights;
    a.out = out;
    return record_cuda_error(
        launch_combine(y_dtype == FP4Q_OUT_F32, out_dtype == FP4Q_OUT_F32, rot, a, stream));
}

fp4q_status fp4q_expert_combine_bwd(const void* g, fp4q_dtype g_dtype, const void* y,
                                    fp4q_dtype y_dtype, int64_t rows, int64_t cols,
                                    const int32_t* slots, int64_t tokens, int k,
                                    const float* weights, void* dy, float* dweights,
                                    cudaStream_t stream)
{
    if (!valid_dtype(g_dtype) || !valid_dtype(y_dtype))
        return FP4Q_ERR_UNSUPPORTED;
    if (k < 1 || k > FP4Q_MAX_CHOICES || !valid_size(rows, cols) || !valid_size(tokens, cols) ||
        cols % 8 != 0)
        return FP4Q_ERR_SHAPE;
    if (tokens == 0 || cols == 0)
        return FP4Q_OK;
    if (g == nullptr || slots == nullptr || (rows > 0 && dy == nullptr) ||
        (rows > 0 && dweights != nullptr && y == nullptr))
        return FP4Q_ERR_NULL;
    if (misaligned(g, 16) || misaligned(y, 16) || misaligned(dy, 16) || misaligned(slots, 4) ||
        misaligned(weights, 4) || misaligned(dweights, 4))
        return FP4Q_ERR_ALIGN;
    if (cudaError_t ie = injected_launch_error())
        return record_cuda_error(ie);
    CombineBwdArgs a;
    a.g = g;
    a.y = y;
    a.rows = rows;
    a.cols = cols;
    a.slots = slots;
    a.tokens = tokens;
    a.k = k;
    a.weights = weights;
    a.dy = dy;
    a.dw = dweights;
    return record_cuda_error(
        launch_combine_bwd(g_dtype == FP4Q_OUT_F32, y_dtype == FP4Q_OUT_F32, a, stream));
}

}  // extern "C"

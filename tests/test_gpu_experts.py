"""The mixture-of-experts entry points on the GPU: the sort by expert against
its definition, quantized rows bit for bit against the oracle, the grouped
product within the fp32 summation bound, combine and the gradients within the
rounding of their types, and a whole layer, also captured and replayed."""
import numpy as np
import pytest
import torch

import expert_ref as ref
from microscaling_fp4_quantization_bf16_b200 import synth

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24   # half a step of fp32, relative
UBF = 2.0 ** -8    # of bf16
PAD8 = 0xA5


def plan_of(gpu, ids, experts, dtype=torch.int64, **kw):
    return gpu.expert_sort(torch.from_numpy(ids).to(dtype).cuda(), experts, **kw)


def filled(shape, dtype):
    """A buffer whose bytes all read 0xA5: what a call leaves alone still does."""
    n = torch.empty(0, dtype=dtype).element_size()
    t = torch.full((int(np.prod(shape)) * n,), PAD8, dtype=torch.uint8, device="cuda")
    return t.view(dtype).reshape(shape)


def untouched(t, rows_used):
    """Rows of t outside rows_used still hold the fill."""
    b = t.contiguous().view(torch.uint8).reshape(t.shape[0], -1).cpu().numpy()
    keep = np.ones(t.shape[0], bool)
    keep[rows_used] = False
    return (b[keep] == PAD8).all()


# ---------------------------------------------------------------- sort

@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,experts,drop", [
    (1, 1, 1, 0), (1, 8, 64, 0), (33, 2, 8, 0.3), (0, 2, 8, 0), (64, 1, 1024, 0), (511, 8, 7, 0.1),
    (512, 8, 256, 0), (513, 8, 256, 0.05), (1024, 8, 256, 0), (1025, 8, 256, 0.05), (3001, 5, 60, 0), (70000, 3, 128, 0.02),
    (400000, 4, 1024, 0.01), (9000, 1, 1, 1.0)])
def test_sort(gpu, dtype, tokens, k, experts, drop):
    ids = ref.route(tokens, k, experts, tokens + k, drop)
    if tokens > 100:
        ids[5, 0], ids[6, 0] = experts, 2 ** 31 - 1          # no such expert: dropped
        ids[7] = ids[7, 0]                                   # the same expert in every choice
    p = plan_of(gpu, ids, experts, dtype)
    counts, starts, slots = ref.sort(ids, experts)
    assert np.array_equal(p.counts.cpu().numpy(), counts)
    assert np.array_equal(p.starts.cpu().numpy(), starts)
    assert np.array_equal(p.slots.cpu().numpy(), slots)
    assert p.rows == gpu.expert_rows(tokens * k, experts) and p.rows >= starts[-1]


def test_sort_one_expert_takes_all(gpu):
    ids = np.full((20000, 2), 3)
    p = plan_of(gpu, ids, 16)
    counts, starts, slots = ref.sort(ids, 16)
    assert np.array_equal(p.slots.cpu().numpy(), slots)
    assert np.array_equal(p.starts.cpu().numpy(), starts)


def test_sort_into_given_buffers_on_another_stream(gpu):
    ids = ref.route(700, 4, 32, 1, 0.1)
    side = torch.cuda.Stream()
    t = torch.from_numpy(ids).cuda()
    first = gpu.expert_sort(t, 32)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        second = gpu.expert_sort(t, 32, out=gpu.ExpertPlan(
            torch.empty_like(first.counts), torch.empty_like(first.starts),
            torch.empty_like(first.slots), first.rows + 128))
    side.synchronize()
    assert torch.equal(first.slots, second.slots) and torch.equal(first.starts, second.starts)


# ---------------------------------------------------------------- quantized rows

def check_rows(q, want, rows_of, cols, fmt, dq_dtype):
    """Quantized q holds, at row r of each (source row, r) pair, the oracle's `want` of the source row."""
    src, dst = rows_of
    codes = q.codes.cpu().numpy()
    assert np.array_equal(codes[dst], want["codes"][src])
    assert untouched(q.codes, dst)
    blocks = cols // ref.BLOCK[fmt]
    sc = ref.mma_rows(q.scales.cpu().numpy(), q.codes.shape[0], blocks)
    assert np.array_equal(sc[dst, :blocks], want["scales"][src])
    assert (sc[dst, blocks:] == 0).all()                     # padding blocks of written rows
    rest = np.ones(sc.shape[0], bool)
    rest[dst] = False
    assert (sc[rest] == PAD8).all()
    if fmt == "nvfp4":
        assert np.float32(q.global_scale.item()) == np.float32(want["global_scale"])
    if dq_dtype is not None:
        dq = torch.from_numpy(want["dq"]).to(dq_dtype).view(torch.uint8).numpy()
        got = q.dq.view(torch.uint8).cpu().numpy()
        assert np.array_equal(got[dst], dq.reshape(dq.shape[0], -1)[src])
        assert untouched(q.dq, dst)


def buffers(gpu, rows, cols, fmt, dq_dtype):
    from microscaling_fp4_quantization_bf16_b200 import experts as ex
    return gpu.Quantized(filled((rows, cols // 2), torch.uint8),
                         filled((ex.scale_bytes(rows, cols, fmt),), torch.uint8),
                         torch.empty(1, device="cuda") if fmt == "nvfp4" else None, None,
                         filled((rows, cols), dq_dtype) if dq_dtype is not None else None)


QUANTS = [("nvfp4", s, r) for s in ("absmax", "prevent_zero", "four_over_six") for r in (0, 16, 128)]
QUANTS += [("nvfp4", "four_over_six", 32), ("nvfp4", "absmax", 64), ("nvfp4", "brute_force", 0),
           ("mxfp4", "brute_force", 32)] + [("mxfp4", "absmax", r) for r in (0, 16, 32, 64, 128)]


@pytest.mark.parametrize("fmt,strategy,rot", QUANTS)
def test_quantize_rows(gpu, fmt, strategy, rot):
    tokens, k, experts, cols = 77, 3, 9, 384
    x = synth.laplace_outliers(tokens, cols, seed=rot + 1)
    ids = ref.route(tokens, k, experts, 3, 0.1)
    p = plan_of(gpu, ids, experts)
    q = gpu.expert_quantize(x.cuda(), p, fmt, strategy, rot, out=buffers(gpu, p.rows, cols, fmt, torch.bfloat16))
    slots = p.slots.cpu().numpy()
    src, j = np.nonzero(slots >= 0)
    check_rows(q, ref.quantize(ref.bits(x), fmt, strategy, rot), (src, slots[src, j]), cols, fmt, torch.bfloat16)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens,k,experts,cols,dq", [
    (1, 1, 1, 32, torch.float32), (1, 8, 64, 1056, torch.bfloat16), (5, 2, 3, 96, torch.float32),
    (300, 1, 4, 160, None), (129, 64, 1024, 64, torch.bfloat16), (1000, 2, 2, 4064, torch.float32),
    (7, 40, 64, 2048, torch.bfloat16)])
def test_quantize_shapes(gpu, fmt, tokens, k, experts, cols, dq):
    x = synth.laplace_outliers(tokens, cols, seed=cols)
    ids = ref.route(tokens, k, experts, cols, 0.02)
    p = plan_of(gpu, ids, experts)
    amax = torch.full((1,), 30.0, device="cuda") if tokens % 2 and fmt == "nvfp4" else None
    q = gpu.expert_quantize(x.cuda(), p, fmt, "absmax", 0, amax, out=buffers(gpu, p.rows, cols, fmt, dq))
    slots = p.slots.cpu().numpy()
    src, j = np.nonzero(slots >= 0)
    want = ref.quantize(ref.bits(x), fmt, "absmax", 0, None if amax is None else 30.0)
    check_rows(q, want, (src, slots[src, j]), cols, fmt, dq)


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("fmt,strategy,rot", QUANTS)
def test_glu_rows(gpu, fmt, strategy, rot, act):
    tokens, k, experts, cols = 50, 2, 5, 384
    ids = ref.route(tokens, k, experts, 4, 0.1)
    p = plan_of(gpu, ids, experts)
    gu = synth.gaussian(p.rows, 2 * cols, seed=rot + 7, std=2.0)
    q = gpu.glu_quantize(gu.cuda(), fmt, strategy, rot, p, act, out=buffers(gpu, p.rows, cols, fmt, torch.float32))
    slots = p.slots.cpu().numpy().reshape(-1)
    dst = slots[slots >= 0]
    h = ref.glu(ref.bits(gu)[dst], act)
    check_rows(q, ref.quantize(h, fmt, strategy, rot), (np.arange(dst.size), dst), cols, fmt, torch.float32)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (130, 1056), (600, 2048)])
def test_glu_all_rows(gpu, fmt, rows, cols):
    """Without a plan: every row, any number of them."""
    gu = synth.gaussian(rows, 2 * cols, seed=rows, std=1.5)
    amax = torch.full((1,), 9.0, device="cuda") if rows % 2 and fmt == "nvfp4" else None
    q = gpu.glu_quantize(gu.cuda(), fmt, "absmax", 0, None, "silu", amax, out=buffers(gpu, rows, cols, fmt, torch.bfloat16))
    h = ref.glu(ref.bits(gu), "silu")
    want = ref.quantize(h, fmt, "absmax", 0, None if amax is None else 9.0)
    blocks = cols // ref.BLOCK[fmt]
    assert np.array_equal(q.codes.cpu().numpy(), want["codes"])
    assert np.array_equal(ref.mma_rows(q.scales.cpu().numpy(), rows, blocks)[:, :blocks], want["scales"])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("scale", [1.0, 3.0, 2.0 ** -60])
def test_glu_every_gate(gpu, act, scale):
    """Every finite bf16 gate up to 2^14 in magnitude against eight values: the
    rounding of h decides the codes, so equal codes need h's own bits."""
    g = np.concatenate([np.arange(0, 0x4680, dtype=np.uint16), np.arange(0x8000, 0xC680, dtype=np.uint16)])
    g = np.resize(g, -(-g.size // 32) * 32)
    rng = np.random.default_rng(5)
    g = np.stack([rng.permutation(g) for _ in range(8)])
    u = ref.bits((torch.from_numpy(rng.standard_normal(g.shape)) * scale).to(torch.bfloat16))
    gu = np.concatenate([g, u], 1)
    # one gate to a block of otherwise equal magnitude would hide in its scale: quantize with blocks as they come
    t = torch.from_numpy(gu.view(np.int16)).view(torch.bfloat16).cuda()
    q = gpu.glu_quantize(t, "mxfp4", "absmax", 0, None, act, dq_dtype=torch.float32)
    want = ref.quantize(ref.glu(gu, act), "mxfp4", "absmax", 0)
    assert np.array_equal(q.codes.cpu().numpy(), want["codes"])
    assert np.array_equal(q.dq.cpu().numpy(), want["dq"])


def test_empty_calls(gpu):
    p = plan_of(gpu, np.zeros((0, 2), np.int64), 4)
    assert p.rows == 0 and p.starts.tolist() == [0] * 5 and p.counts.tolist() == [0] * 4
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    q = gpu.expert_quantize(x, p, "nvfp4")
    assert q.codes.shape == (0, 32) and q.global_scale.item() == 1.0
    w = gpu.expert_weights(synth.gaussian(4 * 16, 64, seed=1).reshape(4, 16, 64).cuda(), "nvfp4")
    d = gpu.expert_gemm(q.codes, q.scales, q.global_scale, w.codes, w.scales, w.global_scale, p)
    assert d.shape == (0, 16)
    assert gpu.expert_combine(d, p).shape == (0, 16)
    dy, dw = gpu.expert_combine_bwd(torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), d, p)
    assert dy.shape == (0, 16) and dw.shape == (0, 2)
    gu = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert gpu.glu_quantize(gu, "nvfp4", plan=p).global_scale.item() == 1.0
    assert gpu.glu_bwd(gu, torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), p).shape == (0, 128)


# ---------------------------------------------------------------- grouped product

def operands(gpu, ids, experts, N, K, fmt, seed, strategy="absmax"):
    p = plan_of(gpu, ids, experts)
    x = synth.laplace_outliers(ids.shape[0], K, seed=seed)
    w = synth.gaussian(experts * N, K, seed=seed + 1, std=0.02).reshape(experts, N, K)
    q = gpu.expert_quantize(x.cuda(), p, fmt, strategy)
    return p, q, gpu.expert_weights(w.cuda(), fmt, strategy)


def check_product(p, q, w, d, fmt, N, K, f32, sample=None):
    counts, starts = p.counts.cpu().numpy(), p.starts.cpu().numpy()
    codes = q.codes.cpu().numpy()
    a = ref.values(codes, q.scales.cpu().numpy(), p.rows, K, fmt)
    got = d.cpu()
    used = []
    for e, c in enumerate(counts):
        if c == 0:
            continue
        used += list(range(starts[e], starts[e] + c))
        rows = np.arange(starts[e], starts[e] + c)
        if sample is not None and c > sample:
            rows = np.unique(np.concatenate([rows[:3], rows[-3:], np.random.default_rng(e).choice(rows, sample)]))
        b = ref.values(w.codes[e].cpu().numpy(), w.scales[e].cpu().numpy(), N, K, fmt)
        alpha = 1.0
        if fmt == "nvfp4":
            alpha = float(np.float32(q.global_scale.item()) * np.float32(w.global_scale[e].item()))
        want = alpha * (a[rows] @ b.T)
        # fp32 accumulation of K products, one product with alpha, one rounding
        bound = (K + 1) * U24 * abs(alpha) * (np.abs(a[rows]) @ np.abs(b).T)
        if not f32:
            bound = bound + UBF * (np.abs(want) + bound)
        err = np.abs(ref.to64(got[rows]) - want)
        assert (err <= bound + 1e-45).all(), (e, c, (err - bound).max(), np.argwhere(err > bound)[:4])
    return used


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("tokens,k,experts,N,K", [
    (1, 1, 1, 128, 256), (1, 1, 1, 8, 32), (128, 1, 1, 128, 64), (16, 2, 4, 256, 512), (40, 1, 1, 136, 96),
    (200, 2, 3, 264, 1056), (33, 4, 16, 1000, 544), (700, 1, 2, 384, 768), (1500, 2, 5, 512, 288),
    (3, 64, 1024, 16, 128)])
def test_product(gpu, fmt, f32, tokens, k, experts, N, K):
    ids = ref.route(tokens, k, experts, tokens + N, 0.02 if tokens > 30 else 0.0)
    p, q, w = operands(gpu, ids, experts, N, K, fmt, tokens + K)
    out = filled((p.rows, N), torch.float32 if f32 else torch.bfloat16)
    d = gpu.expert_gemm(q.codes, q.scales, q.global_scale, w.codes, w.scales, w.global_scale, p, fmt, out=out)
    torch.cuda.synchronize()
    assert gpu.load().fp4q_device_errors() == 0
    used = check_product(p, q, w, d, fmt, N, K, f32)
    assert untouched(d, used)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("rows", [1, 15, 16, 17, 127, 128, 129, 207, 208, 209, 255, 256, 257, 511, 513, 1000])
def test_product_segment_lengths(gpu, fmt, rows):
    """One long and several short segments, at every edge of the row tiles."""
    experts, N, K = 4, 264, 320
    ids = np.concatenate([np.full(rows, 2), np.full(3, 0), np.full(max(1, rows // 2), 3)])[:, None]
    ids = np.random.default_rng(rows).permutation(ids)
    p, q, w = operands(gpu, ids, experts, N, K, fmt, rows)
    out = filled((p.rows, N), torch.float32)
    d = gpu.expert_gemm(q.codes, q.scales, q.global_scale, w.codes, w.scales, w.global_scale, p, fmt, out=out)
    used = check_product(p, q, w, d, fmt, N, K, True)
    assert untouched(d, used)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_product_many_waves(gpu, fmt):
    """Several tiles a CTA, both accumulators in turn, many stages."""
    experts, N, K = 3, 4096, 2048
    ids = ref.route(3000, 1, experts, 9)
    p, q, w = operands(gpu, ids, experts, N, K, fmt, 9)
    d = gpu.expert_gemm(q.codes, q.scales, q.global_scale, w.codes, w.scales, w.global_scale, p, fmt)
    check_product(p, q, w, d, fmt, N, K, False, sample=12)


def test_product_equals_the_dense_product(gpu):
    """One expert, one choice a token: gemm()'s operands, and its result up to the order of sums."""
    M, N, K = 256, 512, 1024
    x, w = synth.laplace_outliers(M, K, seed=3), synth.gaussian(N, K, seed=4, std=0.02)
    qx, qw = gpu.quantize_mma(x.cuda(), "nvfp4"), gpu.quantize_mma(w.cuda(), "nvfp4")
    dense = gpu.gemm(qx.codes, qx.scales, qx.global_scale, qw.codes, qw.scales, qw.global_scale, "nvfp4", torch.float32)
    p = plan_of(gpu, np.zeros((M, 1), np.int64), 1)
    q = gpu.expert_quantize(x.cuda(), p, "nvfp4", global_amax=gpu.global_amax(x.cuda()))
    assert torch.equal(q.codes[:M], qx.codes) and torch.equal(q.scales[:qx.scales.numel()], qx.scales)
    ew = gpu.expert_weights(w.cuda()[None], "nvfp4")
    assert torch.equal(ew.codes[0], qw.codes) and torch.equal(ew.scales[0], qw.scales)
    d = gpu.expert_gemm(q.codes, q.scales, q.global_scale, ew.codes, ew.scales, ew.global_scale, p, "nvfp4", torch.float32)
    a = ref.values(qx.codes.cpu().numpy(), qx.scales.cpu().numpy(), M, K, "nvfp4")
    b = ref.values(qw.codes.cpu().numpy(), qw.scales.cpu().numpy(), N, K, "nvfp4")
    alpha = qx.global_scale.item() * qw.global_scale.item()
    bound = 2 * (K + 1) * U24 * alpha * (np.abs(a) @ np.abs(b).T)
    assert (np.abs(ref.to64(d[:M]) - ref.to64(dense)) <= bound).all()


def test_product_forms_agree(gpu):
    """One CTA or a pair to a tile, on the same operands (through the C call's mean_rows): both within the fp32 bound."""
    experts, N, K = 5, 392, 608
    p, q, w = operands(gpu, ref.route(900, 2, experts, 4, 0.05), experts, N, K, "nvfp4", 4)
    for mean in (1, 128, 129, 10 ** 6):
        d = filled((p.rows, N), torch.float32)
        st = gpu.load().fp4q_expert_gemm(q.codes.data_ptr(), q.scales.data_ptr(), q.global_scale.data_ptr(),
                                         w.codes.data_ptr(), w.scales.data_ptr(), w.global_scale.data_ptr(),
                                         p.counts.data_ptr(), p.starts.data_ptr(), experts, p.rows, N, K, 0, mean,
                                         d.data_ptr(), 0, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert untouched(d, check_product(p, q, w, d, "nvfp4", N, K, True))


def test_product_leaves_out_bad_segments(gpu):
    """Segments that do not fit the buffer or start off a row tile are not computed."""
    experts, N, K = 4, 64, 128
    ids = ref.route(100, 1, experts, 2)
    p, q, w = operands(gpu, ids, experts, N, K, "mxfp4", 2)
    bad = gpu.ExpertPlan(p.counts.clone(), p.starts.clone(), p.slots, p.rows)
    bad.counts[0] = p.rows + 1
    bad.starts[1] = 64
    bad.counts[2] = -5
    out = filled((p.rows, N), torch.bfloat16)
    d = gpu.expert_gemm(q.codes, q.scales, None, w.codes, w.scales, None, bad, "mxfp4", out=out)
    good = gpu.expert_gemm(q.codes, q.scales, None, w.codes, w.scales, None, p, "mxfp4")
    s, c = int(p.starts[3]), int(p.counts[3])
    assert torch.equal(d[s:s + c], good[s:s + c])
    assert untouched(d, list(range(s, s + c)))


# ---------------------------------------------------------------- combine and gradients

@pytest.mark.parametrize("y32,o32", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("tokens,k,experts,cols,rot,weighted", [
    (1, 1, 1, 8, 0, True), (37, 8, 16, 1032, 0, True), (500, 2, 8, 256, 0, False), (20, 13, 30, 128, 128, False),
    (65, 3, 4, 160, 32, False), (64, 4, 4, 64, 64, True), (33, 2, 5, 48, 16, False)])
def test_combine(gpu, y32, o32, tokens, k, experts, cols, rot, weighted):
    ids = ref.route(tokens, k, experts, cols, 0.15)
    if tokens > 2:
        ids[1] = -1                                     # a token with no choice left
    p = plan_of(gpu, ids, experts)
    y = torch.from_numpy(np.random.default_rng(cols).standard_normal((p.rows, cols))).to(torch.float32 if y32 else torch.bfloat16)
    w = torch.from_numpy(np.random.default_rng(k).random((tokens, k))).float() if weighted else None
    out = gpu.expert_combine(y.cuda(), p, None if w is None else w.cuda(), rot, torch.float32 if o32 else torch.bfloat16)
    slots = p.slots.cpu().numpy()
    y64 = np.where((slots >= 0)[..., None], ref.to64(y)[np.maximum(slots, 0)], 0.0)
    w64 = np.ones((tokens, k)) if w is None else ref.to64(w)
    term = w64[..., None] * y64
    want = ref.rotate(term.sum(1), rot)
    # k fused steps, then log2(rot) butterflies and a factor whose own rounding counts, in fp32; a rotation spreads the
    # error of a chunk over its values (every entry of H is 1 / sqrt(rot) in magnitude)
    size = np.abs(term).sum(1)
    if rot:
        size = np.repeat(size.reshape(-1, rot).sum(1) / np.sqrt(rot), rot).reshape(size.shape)
    bound = (k + np.log2(rot or 1) + 2) * U24 * size * 1.01
    if not o32:
        bound = bound + UBF * (np.abs(want) + bound)
    assert (np.abs(ref.to64(out) - want) <= bound).all()
    if tokens > 2:
        assert (out[1] == 0).all()


@pytest.mark.parametrize("g32,y32", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("tokens,k,experts,cols", [(1, 1, 1, 8), (37, 8, 16, 1032), (100, 2, 8, 4096), (9, 13, 30, 264)])
def test_combine_gradient(gpu, g32, y32, tokens, k, experts, cols):
    ids = ref.route(tokens, k, experts, cols, 0.15)
    p = plan_of(gpu, ids, experts)
    rng = np.random.default_rng(cols + k)
    ty, tg = (torch.float32 if b else torch.bfloat16 for b in (y32, g32))
    y = torch.from_numpy(rng.standard_normal((p.rows, cols))).to(ty)
    g = torch.from_numpy(rng.standard_normal((tokens, cols))).to(tg)
    w = torch.from_numpy(rng.random((tokens, k))).float()
    dy, dw = gpu.expert_combine_bwd(g.cuda(), y.cuda(), p, w.cuda(), out=filled((p.rows, cols), ty))
    slots = p.slots.cpu().numpy()
    t, j = np.nonzero(slots >= 0)
    r = slots[t, j]
    want = ref.to64(w)[t, j][:, None] * ref.to64(g)[t]
    bound = (U24 + (0 if y32 else UBF)) * np.abs(want) * 1.01
    assert (np.abs(ref.to64(dy)[r] - want) <= bound).all()
    assert untouched(dy, r)
    part = ref.to64(g)[t] * ref.to64(y)[r]
    wd = np.zeros((tokens, k))
    wd[t, j] = part.sum(1)
    bd = np.zeros((tokens, k))
    bd[t, j] = U24 * np.abs(part.sum(1)) + cols * 2.0 ** -52 * np.abs(part).sum(1)   # 64 bits, rounded once
    assert (np.abs(dw.double().cpu().numpy() - wd) <= bd).all()
    same, none = gpu.expert_combine_bwd(g.cuda(), y.cuda(), p, w.cuda(), want_dweights=False)
    assert none is None and torch.equal(same[torch.from_numpy(r).cuda()], dy[torch.from_numpy(r).cuda()])


def test_combine_gradient_that_cancels(gpu):
    """A router's gradient that is a millionth of its terms keeps its digits."""
    cols = 4096
    p = plan_of(gpu, np.zeros((1, 1), np.int64), 1)
    rng = np.random.default_rng(3)
    g = torch.from_numpy(rng.standard_normal((1, cols))).to(torch.bfloat16)
    y = torch.zeros(p.rows, cols, dtype=torch.bfloat16)
    y[0] = torch.from_numpy(rng.standard_normal(cols)).to(torch.bfloat16)
    y[0, cols // 2:] = -y[0, :cols // 2] * 1.0
    g[0, cols // 2:] = g[0, :cols // 2]
    y[0, 7] *= 1 + 2.0 ** -7
    want = (ref.to64(g)[0] * ref.to64(y)[0]).sum()
    _, dw = gpu.expert_combine_bwd(g.cuda(), y.cuda(), p)
    assert want != 0 and abs(dw.item() - want) <= U24 * abs(want) + cols * 2.0 ** -52 * cols


def test_combine_gradient_against_differences(gpu):
    """d/dw and d/dy of <g, combine(y, w)>, which is linear in each: a difference of two calls is exact up to rounding."""
    tokens, k, experts, cols = 6, 2, 3, 64
    p = plan_of(gpu, ref.route(tokens, k, experts, 1), experts)
    rng = np.random.default_rng(1)
    y = torch.from_numpy(rng.standard_normal((p.rows, cols))).float().cuda()
    g = torch.from_numpy(rng.standard_normal((tokens, cols))).float().cuda()
    w = torch.from_numpy(rng.random((tokens, k))).float().cuda()
    dy, dw = gpu.expert_combine_bwd(g, y, p, w)

    def loss(y, w):
        return (g.double() * gpu.expert_combine(y, p, w, 0, torch.float32).double()).sum().item()
    base = loss(y, w)
    # each call's outputs are off by (k + 1) half steps of their terms
    noise = 2 * (k + 1) * U24 * float((g.double().abs().sum() * y.abs().max() * 4))
    for t, j in ((0, 0), (3, 1)):
        w2 = w.clone()
        w2[t, j] += 1.0
        assert abs(loss(y, w2) - base - dw[t, j].item()) <= noise
        r = int(p.slots[t, j])
        y2 = y.clone()
        y2[r, 5] += 1.0
        assert abs(loss(y2, w) - base - dy[r, 5].item()) <= noise


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("rows,cols,rot,plan", [(1, 8, 0, False), (50, 1032, 0, True), (40, 128, 128, True),
                                                (33, 96, 32, False), (30, 64, 64, True), (30, 48, 16, False)])
def test_glu_gradient(gpu, act, rows, cols, rot, plan):
    if rot and cols % 32:
        with pytest.raises(gpu.Fp4qError):
            gpu.glu_bwd(torch.zeros(rows, 2 * cols, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda"), None, act, rot)
        return
    p = plan_of(gpu, ref.route(rows, 1, 3, rows, 0.1), 3) if plan else None
    n = p.rows if plan else rows
    gu = synth.gaussian(n, 2 * cols, seed=cols, std=2.5)
    gu[0, :3] = torch.tensor([-95.0, 80.0, 0.0])
    dh = synth.gaussian(n, cols, seed=cols + 1, std=1.0)
    out = gpu.glu_bwd(gu.cuda(), dh.cuda(), p, act, rot, out=filled((n, 2 * cols), torch.bfloat16))
    taken = np.arange(n) if p is None else p.slots.cpu().numpy().reshape(-1)
    taken = taken[taken >= 0]
    g, u = np.split(ref.to64(gu)[taken], 2, axis=1)
    d = ref.rotate(ref.to64(dh)[taken], rot)
    z, dz = ref.gate(g, act)
    s = ref.sigmoid(z)
    dg, du = d * u * (s + g * s * (1 - s) * dz), d * g * s
    want = np.concatenate([dg, du], 1)
    # s is off by 2^-20 + 2^-21 max(-z, 0) relative at most (hardware 2^x and 1/x); every other step by a few half steps. The
    # two terms of a'(g) may cancel, so their magnitudes count. Through a rotation the error of a chunk spreads.
    es = (2.0 ** -20 + 2.0 ** -21 * np.maximum(-z, 0)) + 12 * U24
    size = np.concatenate([np.abs(u) * (s + np.abs(g) * s * dz) * 3, np.abs(g) * s], 1) * np.concatenate([es, es], 1)
    err_d = np.zeros_like(d)
    if rot:
        err_d = (np.log2(rot) + 2) * U24 * np.repeat(np.abs(ref.to64(dh)[taken]).reshape(-1, rot).sum(1) / np.sqrt(rot), rot).reshape(d.shape)
    factor = np.concatenate([np.abs(u) * (s + np.abs(g) * s * dz), np.abs(g) * s], 1)
    bound = size * np.concatenate([np.abs(d)] * 2, 1) + factor * np.concatenate([err_d] * 2, 1)
    bound = (bound + UBF * (np.abs(want) + bound)) * 1.01 + 2.0 ** -120
    assert (np.abs(ref.to64(out)[taken] - want) <= bound).all()
    assert untouched(out, taken)


def test_glu_gradient_against_differences(gpu):
    """The formula itself against central differences of a(g) u in 64 bits."""
    for act in ("silu", "gelu_tanh"):
        g = np.linspace(-6, 6, 64)[None]
        u = np.cos(np.arange(64.0))[None]
        gu = torch.from_numpy(np.concatenate([g, u], 1)).to(torch.bfloat16)
        g, u = np.split(ref.to64(gu), 2, axis=1)
        got = ref.to64(gpu.glu_bwd(gu.cuda(), torch.ones(1, 64, dtype=torch.bfloat16, device="cuda"), None, act))
        f = lambda g, u: g * u * ref.sigmoid(ref.gate(g, act)[0])  # noqa: E731
        h = 1e-5
        want = np.concatenate([(f(g + h, u) - f(g - h, u)) / (2 * h), (f(g, u + h) - f(g, u - h)) / (2 * h)], 1)
        # one bf16 rounding, the fp32 error near a zero of a'(g), and the differences' own h^2 and 2^-53 / h
        assert (np.abs(got - want) <= UBF * np.abs(want) + 2.0 ** -17 * (1 + np.abs(np.concatenate([g, u], 1))) + 1e-9).all()


def test_dispatch_gradient(gpu):
    """expert_combine without weights is the transpose of the dispatch (rotation and copies) in front of the rounding."""
    tokens, k, experts, cols, rot = 40, 3, 6, 256, 64
    p = plan_of(gpu, ref.route(tokens, k, experts, 8, 0.2), experts)
    rng = np.random.default_rng(2)
    x, dy = rng.standard_normal((tokens, cols)), rng.standard_normal((p.rows, cols))
    dx = gpu.expert_combine(torch.from_numpy(dy).float().cuda(), p, None, rot, torch.float32)
    slots = p.slots.cpu().numpy()
    t, j = np.nonzero(slots >= 0)
    lhs = (ref.rotate(x, rot)[t] * dy[slots[t, j]]).sum()          # <dispatch(x), dy>
    rhs = (x * ref.to64(dx)).sum()                                 # <x, dispatch^T(dy)>
    # dx is off by (k + log2 rot + 2) half steps of a chunk's terms, and dy was rounded to fp32 once
    noise = (k + 6 + 4) * U24 * np.abs(x).max() * np.abs(dy).sum() * np.sqrt(rot)
    assert abs(lhs - rhs) <= noise


# ---------------------------------------------------------------- more than 2^31 elements

def big_plan(gpu, tokens, experts=2):
    ids = torch.randint(0, experts, (tokens, 1), generator=torch.Generator().manual_seed(1)).cuda()
    p = gpu.expert_sort(ids, experts)
    slots = p.slots.reshape(-1)
    last = torch.cat([slots.topk(4).indices, slots.topk(3, largest=False).indices, torch.tensor([tokens // 2]).cuda()])
    return p, last, slots[last].long()


def patterned(rows, cols):
    """bf16 [rows, cols] whose rows repeat every 257."""
    base = synth.gaussian(257, cols, seed=3).cuda()
    return base.repeat(-(-rows // 257), 1)[:rows].contiguous()


def test_combine_beyond_32_bits(gpu):
    tokens, cols = 270000, 8192
    p, t, r = big_plan(gpu, tokens)
    y = patterned(p.rows, cols)
    assert y.numel() > 2 ** 31 and int(r.max()) * cols > 2 ** 31
    w = torch.full((tokens, 1), 0.5, device="cuda")
    out = gpu.expert_combine(y, p, w)
    assert torch.equal(out[t], (y[r].float() * 0.5).to(torch.bfloat16))     # exact: a power of two
    dy, dw = gpu.expert_combine_bwd(out, y, p, w, out=y.clone())
    assert torch.equal(dy[r], (out[t].float() * 0.5).to(torch.bfloat16))
    want = (out[t].double() * y[r].double()).sum(1)
    assert ((dw[t, 0].double() - want).abs() <= cols * U24 * (out[t].double() * y[r].double()).abs().sum(1)).all()


def test_quantizers_beyond_32_bits(gpu):
    tokens, cols = 270000, 8192
    p, t, r = big_plan(gpu, tokens)
    x = patterned(tokens, cols)
    q = gpu.expert_quantize(x, p, "mxfp4", "absmax", 32)
    want = ref.quantize(ref.bits(x[t]), "mxfp4", "absmax", 32)
    assert np.array_equal(q.codes[r].cpu().numpy(), want["codes"])
    del x
    gu = patterned(p.rows, 2 * cols)
    q = gpu.glu_quantize(gu, "mxfp4", "absmax", 0, p, out=q)
    want = ref.quantize(ref.glu(ref.bits(gu[r]), "silu"), "mxfp4", "absmax", 0)
    assert np.array_equal(q.codes[r].cpu().numpy(), want["codes"])
    sc = ref.mma_rows(q.scales.cpu().numpy(), p.rows, cols // 32)
    assert np.array_equal(sc[r.cpu().numpy()], want["scales"])
    dh = patterned(p.rows, cols)
    out = gpu.glu_bwd(gu, dh, p)
    few = gpu.glu_bwd(gu[r].contiguous(), dh[r].contiguous())
    assert torch.equal(out[r], few)


def test_product_beyond_32_bits(gpu):
    tokens, N, K = 140000, 16384, 64
    p, t, r = big_plan(gpu, tokens)
    q = gpu.expert_quantize(patterned(tokens, K), p, "mxfp4")
    w = gpu.expert_weights(patterned(2 * N, K).reshape(2, N, K), "mxfp4")
    d = gpu.expert_gemm(q.codes, q.scales, None, w.codes, w.scales, None, p, "mxfp4")
    assert int(r.max()) * N > 2 ** 31
    starts = p.starts.tolist()
    a = ref.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), p.rows, K, "mxfp4")
    for row in r.tolist():
        e = 0 if row < starts[1] else 1
        b = ref.values(w.codes[e].cpu().numpy(), w.scales[e].cpu().numpy(), N, K, "mxfp4")
        want = b @ a[row]
        bound = (K + 1) * U24 * (np.abs(b) @ np.abs(a[row]))
        assert (np.abs(ref.to64(d[row]) - want) <= bound + UBF * (np.abs(want) + bound)).all()


# ---------------------------------------------------------------- refusals

def test_refusals(gpu):
    """Arguments that do not belong together raise before anything runs."""
    p = plan_of(gpu, ref.route(20, 2, 4, 1), 4)
    x = torch.zeros(20, 64, dtype=torch.bfloat16, device="cuda")
    q = gpu.expert_quantize(x, p, "mxfp4")
    w = gpu.expert_weights(torch.zeros(4, 32, 64, dtype=torch.bfloat16, device="cuda"), "mxfp4")
    y = torch.zeros(p.rows, 64, dtype=torch.bfloat16, device="cuda")
    wt = torch.zeros(20, 2, device="cuda")
    mm = lambda **k: gpu.expert_gemm(k.get("a", q.codes), k.get("sa", q.scales), None, k.get("w", w.codes),  # noqa: E731
                                     k.get("sw", w.scales), None, k.get("p", p), "mxfp4", out=k.get("out"))
    bad = [
        lambda: gpu.expert_sort(torch.zeros(4, 2, dtype=torch.int16, device="cuda"), 4),
        lambda: gpu.expert_sort(torch.zeros(4, dtype=torch.int32, device="cuda"), 4),
        lambda: gpu.expert_sort(torch.zeros(2, 4, dtype=torch.int32, device="cuda").t(), 4),
        lambda: gpu.expert_sort(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 0),
        lambda: gpu.expert_sort(torch.zeros(200, 2, dtype=torch.int32, device="cuda"), 4, rows=128),
        lambda: gpu.expert_sort(torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 4, rows=1000),
        lambda: gpu.expert_quantize(x.float(), p),
        lambda: gpu.expert_quantize(x[:19], p),
        lambda: gpu.expert_quantize(x[:, :48].contiguous(), p),
        lambda: gpu.expert_quantize(x, p, "ue5m3"),
        lambda: gpu.expert_quantize(x, p, "mxfp4", "four_over_six"),
        lambda: gpu.expert_quantize(x, p, "nvfp4", rot=128),
        lambda: gpu.expert_quantize(x, p, "nvfp4", global_amax=torch.zeros(2, device="cuda")),
        lambda: gpu.expert_quantize(x, p, "mxfp4", out=gpu.Quantized(q.codes[:128], q.scales, None, None, None)),
        lambda: mm(a=q.codes[:, :16].contiguous()),
        lambda: mm(sa=q.scales[:-1]),
        lambda: mm(w=w.codes[:3]),
        lambda: mm(sw=w.scales[:, :512].contiguous()[:2]),
        lambda: mm(out=torch.zeros(p.rows, 40, dtype=torch.bfloat16, device="cuda")),
        lambda: mm(out=torch.zeros(p.rows, 32, dtype=torch.float16, device="cuda")),
        lambda: gpu.expert_gemm(q.codes, q.scales, None, w.codes, w.scales, None, p, "nvfp4"),
        lambda: gpu.expert_weights(torch.zeros(4, 32, 40, dtype=torch.bfloat16, device="cuda")),
        lambda: gpu.glu_quantize(y[:, :63].contiguous()),
        lambda: gpu.glu_quantize(y[:100], plan=p),
        lambda: gpu.glu_quantize(y, act="relu"),
        lambda: gpu.glu_bwd(y, y, p),
        lambda: gpu.expert_combine(y[:128], p),
        lambda: gpu.expert_combine(y, p, wt[:, :1].contiguous()),
        lambda: gpu.expert_combine(y, p, wt.double()),
        lambda: gpu.expert_combine(y, p, rot=48),
        lambda: gpu.expert_combine_bwd(x[:, :32].contiguous(), y, p),
        lambda: gpu.expert_combine_bwd(x, y, p, out=torch.zeros_like(y, dtype=torch.float32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, gpu.Fp4qError)):
            call()
            raise AssertionError(f"call {i} was accepted")
    torch.cuda.synchronize()


# ---------------------------------------------------------------- a whole layer

def layer(gpu, x, p, weights, up, down, fmt, rot, amaxes=(None, None)):
    qa = gpu.expert_quantize(x, p, fmt, "absmax", rot, amaxes[0])
    gu = gpu.expert_gemm(qa.codes, qa.scales, qa.global_scale, up.codes, up.scales, up.global_scale, p, fmt)
    qh = gpu.glu_quantize(gu, fmt, "absmax", rot, p, "silu", amaxes[1])
    y = gpu.expert_gemm(qh.codes, qh.scales, qh.global_scale, down.codes, down.scales, down.global_scale, p, fmt)
    return gpu.expert_combine(y, p, weights), gu, y


@pytest.mark.parametrize("fmt,rot", [("nvfp4", 16), ("mxfp4", 128)])
@pytest.mark.parametrize("tokens", [1, 50, 900])
def test_layer(gpu, fmt, rot, tokens):
    """Against the same layer from the dense entry points, expert by expert."""
    k, experts, H, I = 2, 4, 256, 384
    x = synth.laplace_outliers(tokens, H, seed=tokens).cuda()
    wu = synth.gaussian(experts * 2 * I, H, seed=1, std=0.05).reshape(experts, 2 * I, H).cuda()
    wd = synth.gaussian(experts * H, I, seed=2, std=0.05).reshape(experts, H, I).cuda()
    ids = ref.route(tokens, k, experts, tokens, 0.05 if tokens > 1 else 0)
    p = plan_of(gpu, ids, experts)
    weights = torch.rand(tokens, k, generator=torch.Generator().manual_seed(3)).cuda()
    up, down = gpu.expert_weights(wu, fmt, "absmax", rot), gpu.expert_weights(wd, fmt, "absmax", rot)
    calib = [torch.full((1,), v, device="cuda") for v in (80.0, 60.0)] if fmt == "nvfp4" else [None, None]
    out, gu, y = layer(gpu, x, p, weights, up, down, fmt, rot, calib)
    slots = p.slots.cpu().numpy()
    for e in range(experts):
        t, j = np.nonzero(slots * 0 + (ids == e))
        if t.size == 0:
            continue
        r = torch.from_numpy(slots[t, j].astype(np.int64)).cuda()
        qa = gpu.quantize_mma(x[torch.from_numpy(t).cuda()].contiguous(), fmt, "absmax", rot, calib[0])
        uq = gpu.quantize_mma(wu[e].contiguous(), fmt, "absmax", rot)
        want = gpu.gemm(qa.codes, qa.scales, qa.global_scale, uq.codes, uq.scales, uq.global_scale, fmt)
        # the same codes and scales, so fp32 sums in another order, then one rounding each. Both are within (H + 1) half
        # steps of sum |a b|, which is below 600 for these inputs (|x| < 15, the rows of the weights sum to about 10).
        diff = (gu[r].float() - want.float()).abs()
        assert (diff <= 2 * UBF * want.float().abs() + (H + 1) * 2 * U24 * 600).all()
        # from the layer's own gate and value on, bit for bit what the unfused steps give
        h = torch.from_numpy(ref.glu(ref.bits(gu[r].contiguous()), "silu").view(np.int16)).view(torch.bfloat16).cuda()
        qh = gpu.quantize_mma(h, fmt, "absmax", rot, calib[1])
        dq = gpu.quantize_mma(wd[e].contiguous(), fmt, "absmax", rot)
        want = gpu.gemm(qh.codes, qh.scales, qh.global_scale, dq.codes, dq.scales, dq.global_scale, fmt)
        diff = (y[r].float() - want.float()).abs()
        assert (diff <= 2 * UBF * want.float().abs() + (I + 1) * 2 * U24 * 600).all()
    t, j = np.nonzero(slots >= 0)
    total = np.zeros((tokens, k, H))
    total[t, j] = ref.to64(y[torch.from_numpy(slots[t, j].astype(np.int64)).cuda()]) * ref.to64(weights)[t, j][:, None]
    bound = (k + 1) * U24 * np.abs(total).sum(1)
    bound = bound + UBF * (np.abs(total.sum(1)) + bound)
    assert (np.abs(ref.to64(out) - total.sum(1)) <= bound).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_layer_captured_and_replayed(gpu, fmt):
    """Sort and layer in one CUDA graph, replayed with other tokens and another routing; two graphs in turn."""
    tokens, k, experts, H, I = 64, 2, 8, 256, 128
    up = gpu.expert_weights(synth.gaussian(experts * 2 * I, H, seed=1, std=0.05).reshape(experts, 2 * I, H).cuda(), fmt)
    down = gpu.expert_weights(synth.gaussian(experts * H, I, seed=2, std=0.05).reshape(experts, H, I).cuda(), fmt)
    x = torch.empty(tokens, H, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(tokens, k, dtype=torch.int64, device="cuda")
    w = torch.empty(tokens, k, device="cuda")

    def fill(seed):
        x.copy_(synth.laplace_outliers(tokens, H, seed=seed))
        ids.copy_(torch.from_numpy(ref.route(tokens, k, experts, seed, 0.1)))
        w.copy_(torch.rand(tokens, k, generator=torch.Generator().manual_seed(seed)))

    def step():
        return layer(gpu, x, gpu.expert_sort(ids, experts), w, up, down, fmt, 0)[0]
    fill(0)
    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for seed in (1, 2, 3):
        fill(seed)
        want = step()
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out, want)
    assert gpu.load().fp4q_device_errors() == 0


def test_layers_on_two_streams(gpu):
    """Two layers (one of long segments, one of short) on streams of their own, at the same time and with dense
    products between them: each gives what it gives alone."""
    cases = []
    for tokens, fmt, seed in ((900, "nvfp4", 1), (40, "mxfp4", 2)):
        k, experts, H, I = 2, 4, 512, 384
        up = gpu.expert_weights(synth.gaussian(experts * 2 * I, H, seed=seed, std=0.05).reshape(experts, 2 * I, H).cuda(), fmt)
        down = gpu.expert_weights(synth.gaussian(experts * H, I, seed=seed + 5, std=0.05).reshape(experts, H, I).cuda(), fmt)
        x = synth.laplace_outliers(tokens, H, seed=seed).cuda()
        ids = torch.from_numpy(ref.route(tokens, k, experts, seed)).cuda()
        w = torch.rand(tokens, k, generator=torch.Generator().manual_seed(seed)).cuda()
        q = gpu.quantize_mma(x, fmt)

        def run(fmt=fmt, up=up, down=down, x=x, ids=ids, w=w, q=q, experts=experts):
            out = layer(gpu, x, gpu.expert_sort(ids, experts), w, up, down, fmt, 0)[0]
            gs = None if fmt == "mxfp4" else up.global_scale[:1]
            return out, gpu.gemm(q.codes, q.scales, q.global_scale, up.codes[0], up.scales[0], gs, fmt)
        cases.append(run)
    want = [run() for run in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(20):
        for run, stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                got.append(run())
    torch.cuda.synchronize()
    for i, (out, dense) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(dense, want[i % 2][1]), i
    assert gpu.load().fp4q_device_errors() == 0


def test_results_repeat(gpu):
    """The same call twice gives the same bits, products and gradients too."""
    tokens, k, experts, H, N = 3000, 4, 16, 512, 512
    ids = ref.route(tokens, k, experts, 5, 0.05)
    p, q, w = operands(gpu, ids, experts, N, H, "nvfp4", 5)
    run = lambda: gpu.expert_gemm(q.codes, q.scales, q.global_scale, w.codes, w.scales, w.global_scale, p,  # noqa: E731
                                  out=torch.zeros(p.rows, N, dtype=torch.bfloat16, device="cuda"))
    first = run()
    g = synth.gaussian(tokens, N, seed=1).cuda()
    wt = torch.rand(tokens, k, device="cuda")
    one = gpu.expert_combine_bwd(g, first, p, wt, out=torch.zeros_like(first))
    for _ in range(3):
        assert torch.equal(run(), first)
        two = gpu.expert_combine_bwd(g, first, p, wt, out=torch.zeros_like(first))
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])

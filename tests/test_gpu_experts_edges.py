"""The mixture-of-experts entry points on the GPU at the edges of what they allow: the largest and smallest
sizes of a launch, values at the ends of their types' range, empty plans, calls next to each other."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import expert_ref as ref
from microscaling_fp4_quantization_bf16_b200.experts import scale_bytes
from test_gpu_experts import U24, UBF, check_product, filled, operands, untouched

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- grouped product

@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("K", [32, 256, 1024, 1312])
def test_products_in_close_succession(gpu, fmt, K):
    """Products of one short tile a CTA, fewer stages than there are and more, launch after launch: nothing of one is
    left over (a barrier's arrival, a copy) when the next one takes its memory."""
    experts, N = 3, 264                                      # an odd number of output tiles: half a pair has none
    p, q, w = operands(gpu, ref.route(330, 1, experts, K, 0.02), experts, N, K, fmt, K)
    stream = torch.cuda.current_stream().cuda_stream

    def product(mean, d):
        one = gpu.load().fp4q_expert_gemm(
            q.codes.data_ptr(), q.scales.data_ptr(), q.global_scale.data_ptr() if fmt == "nvfp4" else None,
            w.codes.data_ptr(), w.scales.data_ptr(), w.global_scale.data_ptr() if fmt == "nvfp4" else None,
            p.counts.data_ptr(), p.starts.data_ptr(), experts, p.rows, N, K, 1 if fmt == "mxfp4" else 0, mean,
            d.data_ptr(), 0, stream)
        assert one == 0
        return d
    first = {m: product(m, filled((p.rows, N), torch.float32)) for m in (1000, 1)}
    for d in first.values():
        assert untouched(d, check_product(p, q, w, d, fmt, N, K, True))
    again = [(m, product(m, filled((p.rows, N), torch.float32))) for _ in range(100) for m in (1000, 1000, 1)]
    torch.cuda.synchronize()
    for m, d in again:
        assert torch.equal(d.view(torch.int32), first[m].view(torch.int32))
    assert gpu.load().fp4q_device_errors() == 0


# ---------------------------------------------------------------- sort

SORTS_NEAR_48K = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np, torch
import expert_ref as ref
import microscaling_fp4_quantization_bf16_b200 as fp4q
for tokens, k, experts in ((928, 1, 384), (66, 10, 512), (400, 1, 768), (288, 1, 1024), (1000, 1, 351), (4096, 1, 351)):
    ids = ref.route(tokens, k, experts, tokens, 0.05)
    p = fp4q.expert_sort(torch.from_numpy(ids).to(torch.{dtype}).cuda(), experts)
    counts, starts, slots = ref.sort(ids, experts)
    assert np.array_equal(p.counts.cpu().numpy(), counts) and np.array_equal(p.starts.cpu().numpy(), starts)
    assert np.array_equal(p.slots.cpu().numpy(), slots), (tokens, k, experts)
print("sorted")
"""


@pytest.mark.parametrize("dtype", ["int32", "int64"])
def test_sorts_whose_shared_memory_is_near_the_default_limit(gpu, dtype):
    """(warps + 3) experts words just under 48 KB, with the static word above it, in a process that has sorted nothing
    larger before (a larger sort raises the kernel's limit)."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = SORTS_NEAR_48K.format(root=os.path.dirname(here), tests=here, dtype=dtype)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "sorted" in r.stdout, r.stderr[-2000:]


def test_sorts_of_two_threads(gpu):
    """Two host threads that sort among different numbers of experts, each on a stream of its own: no call takes
    another's launch limits."""
    cases = []
    for tokens, experts in ((4096, 1024), (4096, 384)):
        ids = ref.route(tokens, 1, experts, experts, 0.02)
        cases.append((torch.from_numpy(ids).cuda(), experts, torch.from_numpy(ref.sort(ids, experts)[2]).int().cuda()))
    torch.cuda.synchronize()
    wrong = []

    def work(ids, experts, slots):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                out = gpu.expert_sort(ids, experts)
                for _ in range(3000):
                    gpu.expert_sort(ids, experts, out=out)
                torch.cuda.current_stream().synchronize()
                if not torch.equal(out.slots, slots):
                    wrong.append(experts)
        except Exception as e:
            wrong.append(e)
    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


# ---------------------------------------------------------------- a plan without tokens

@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("calibrated", [False, True])
def test_plan_without_tokens_takes_no_row(gpu, fmt, calibrated):
    """A batch without a token in buffers of a fixed size: no row holds a choice, so none is read or written."""
    rows, cols = 256, 64
    p = gpu.expert_sort(torch.empty(0, 2, dtype=torch.int64, device="cuda"), 4, rows=rows)
    assert p.rows == rows and p.starts.tolist() == [0] * 5
    gu = torch.full((rows, 2 * cols), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = gpu.Quantized(filled((rows, cols // 2), torch.uint8), filled((scale_bytes(rows, cols, fmt),), torch.uint8),
                      torch.zeros(1, device="cuda") if fmt == "nvfp4" else None, None, filled((rows, cols), torch.float32))
    amax = torch.full((1,), 5.0, device="cuda") if calibrated else None
    gpu.glu_quantize(gu, fmt, plan=p, global_amax=amax, out=q)
    assert untouched(q.codes, []) and untouched(q.dq, []) and untouched(q.scales[:, None], [])
    assert fmt == "mxfp4" or q.global_scale.item() == 1.0
    out = filled((rows, 2 * cols), torch.bfloat16)
    gpu.glu_bwd(gu, torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda"), p, out=out)
    assert untouched(out, [])
    # and without a plan all rows are taken, as before
    ones = torch.ones(3, 2 * cols, dtype=torch.bfloat16, device="cuda")
    assert (gpu.glu_quantize(ones, fmt, dq_dtype=torch.float32).dq != 0).all()
    # the layer's other calls on such a plan
    x = torch.empty(0, cols, dtype=torch.bfloat16, device="cuda")
    gpu.expert_quantize(x, p, fmt, global_amax=amax, out=q)
    assert untouched(q.codes, []) and untouched(q.dq, []) and untouched(q.scales[:, None], [])
    w = gpu.expert_weights(torch.ones(4, 16, cols, dtype=torch.bfloat16, device="cuda"), fmt)
    d = filled((rows, 16), torch.bfloat16)
    gpu.expert_gemm(q.codes, q.scales, q.global_scale, w.codes, w.scales, w.global_scale, p, fmt, out=d)
    assert untouched(d, [])
    assert gpu.expert_combine(d, p).shape == (0, 16)
    dy, dw = gpu.expert_combine_bwd(torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), d, p, out=filled((rows, 16), torch.bfloat16))
    assert untouched(dy, []) and dw.shape == (0, 2)


# ---------------------------------------------------------------- gradients at the ends of the types' range

def glu_gradient_bound(g, u, d, act):
    """64-bit gradient [dg, du] and the bound of glu_bwd's fp32 steps: s off by 2^-20 + 2^-21 max(-z, 0) relative (hardware
    2^x and 1/x), every other step by a few half steps; the two terms of a'(g) may cancel, so their magnitudes
    count; one bf16 rounding; s below 2^-126 counts as zero."""
    z, dz = ref.gate(g, act)
    s = ref.sigmoid(z)
    want = np.concatenate([d * u * (s + g * s * (1 - s) * dz), d * g * s], 1)
    es = np.where(s < 2.0 ** -125, 1.0, (2.0 ** -20 + 2.0 ** -21 * np.maximum(-z, 0)) + 12 * U24)
    size = np.concatenate([np.abs(d * u) * (s + np.abs(g) * s * (1 - s) * dz) * 3, np.abs(d * g) * s], 1)
    bound = size * np.concatenate([es, es], 1)
    return want, (bound + UBF * (np.abs(want) + bound)) * 1.01 + 2.0 ** -120


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_glu_gradient_of_far_gates(gpu, act):
    """Gates up to the type's largest: a'(g) is 1 or 0 there, and never a number that is none."""
    g = np.array([1e13, 1e15, 2.0 ** 63, 2.0 ** 64, 1e20, 1e30, 3e38, 3.3895313892515355e38])
    g = np.concatenate([g, -g])[None]
    u = np.tile([0.5, -0.75, 1.0, 2.0 ** -20], 4)[None]
    dh = torch.from_numpy(np.tile([0.5, 0.25, -0.5, 1e-10], 4)[None]).to(torch.bfloat16)
    gu = torch.from_numpy(np.concatenate([g, u], 1)).to(torch.bfloat16)
    got = ref.to64(gpu.glu_bwd(gu.cuda(), dh.cuda(), None, act))
    g, u = np.split(ref.to64(gu), 2, axis=1)
    want, bound = glu_gradient_bound(g, u, ref.to64(dh), act)
    assert np.isfinite(got).all() and (np.abs(got - want) <= bound).all(), got


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_glu_gradient_whose_first_product_overflows(gpu, act):
    """dh u beyond fp32 in front of a small a'(g): the gradient itself is in range."""
    g = np.array([-80.0, -70.0, -60.0, -45.0, -200.0, -3e38, 0.0, -1.0]) if act == "silu" else \
        np.array([-8.5, -8.0, -7.5, -6.5, -20.0, -3e38, 0.0, -1.0])
    d = np.array([1e30, 1e25, -1e24, 1e19, 1e30, 1e30, 1e10, 1e10])
    u = np.array([1e30, -1e30, 1e20, 1e30, 1e30, 1e30, 1e20, 1e20])
    gu = torch.from_numpy(np.concatenate([g, u])[None]).to(torch.bfloat16)
    dh = torch.from_numpy(d[None]).to(torch.bfloat16)
    got = ref.to64(gpu.glu_bwd(gu.cuda(), dh.cuda(), None, act))
    g, u = np.split(ref.to64(gu), 2, axis=1)
    want, bound = glu_gradient_bound(g, u, ref.to64(dh), act)
    assert (np.abs(ref.to64(dh) * u)[0, :6] > 3.4e38).all() and np.isfinite(want).all()
    assert np.isfinite(got).all() and (np.abs(got - want) <= bound).all(), (got, want)


@pytest.mark.parametrize("g32,y32", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("what", ["large", "small", "mixed"])
def test_combine_gradient_beyond_the_products_range(gpu, g32, y32, what):
    """Products of two bf16 numbers that fp32 does not hold, in sums that it does: dweights is summed in 64 bits."""
    cols = 4096
    p = gpu.expert_sort(torch.zeros(1, 1, dtype=torch.int64, device="cuda"), 1)
    g, y = np.ones(cols), np.zeros((p.rows, cols))
    if what == "large":                               # 2^128 and its opposite, and 3 beside them
        g[:4], y[0, :4] = 2.0 ** 64, [2.0 ** 64, -2.0 ** 64, 2.0 ** 80, -2.0 ** 80]
        y[0, 9] = 3.0
        want = 3.0
    elif what == "small":                             # 4096 times 2^-160
        g[:], y[0] = 2.0 ** -80, 2.0 ** -80
        want = 2.0 ** -148
    else:                                             # subnormal products: 2^-140 (1 + 2^-7)^2 each, in 8 of which bits are lost
        g[:], y[0] = 2.0 ** -70 * (1 + 2.0 ** -7), 2.0 ** -70 * (1 + 2.0 ** -7)
        want = cols * 2.0 ** -140 * (1 + 2.0 ** -7) ** 2
    g = torch.from_numpy(g[None]).to(torch.float32 if g32 else torch.bfloat16).cuda()
    y = torch.from_numpy(y).to(torch.float32 if y32 else torch.bfloat16).cuda()
    _, dw = gpu.expert_combine_bwd(g, y, p)
    # every sum of these is exact in 64 bits; one rounding to fp32 (2^-148 is a subnormal that fp32 has)
    assert abs(dw.item() - want) <= max(U24 * want, 2.0 ** -150), (dw.item(), want)


def test_combine_gradient_of_infinities(gpu):
    """An infinity or NaN in a row of y comes out in its own choice's gradient and in no other."""
    cols = 512
    p = gpu.expert_sort(torch.tensor([[0, 1, 2, 3]], device="cuda"), 4)
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.ones(p.rows, cols, dtype=dtype, device="cuda")
        r = p.slots[0].tolist()
        y[r[0], 3], y[r[1], 300], y[r[2], 511] = float("inf"), float("-inf"), float("nan")
        dy, dw = gpu.expert_combine_bwd(torch.ones(1, cols, dtype=dtype, device="cuda"), y, p)
        assert dw[0, 0] == float("inf") and dw[0, 1] == float("-inf") and dw[0, 2].isnan() and dw[0, 3] == cols
        assert (dy[p.slots[0].long()] == 1).all()


# ---------------------------------------------------------------- refusals

def test_refused_output_types_and_no_experts(gpu):
    """Types that no output has and weights of no expert raise as the other arguments do, before anything runs."""
    p = gpu.expert_sort(torch.zeros(4, 2, dtype=torch.int64, device="cuda"), 4)
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(p.rows, 64, dtype=torch.bfloat16, device="cuda")
    q = gpu.expert_quantize(x, p, "mxfp4")
    w = gpu.expert_weights(torch.zeros(4, 32, 64, dtype=torch.bfloat16, device="cuda"), "mxfp4")
    none = gpu.ExpertPlan(p.counts[:0], p.starts[:1], p.slots, p.rows)
    for call in (lambda: gpu.expert_quantize(x, p, "mxfp4", dq_dtype=torch.float16),
                 lambda: gpu.glu_quantize(x, "mxfp4", dq_dtype=torch.float64),
                 lambda: gpu.expert_combine(y, p, out_dtype=torch.float16),
                 lambda: gpu.expert_gemm(q.codes, q.scales, None, w.codes, w.scales, None, p, "mxfp4", torch.float16),
                 lambda: gpu.expert_gemm(q.codes, q.scales, None, w.codes[:0], w.scales[:0], None, none, "mxfp4")):
        with pytest.raises(ValueError):
            call()

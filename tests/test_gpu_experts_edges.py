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
from test_gpu_experts import check_product, filled, operands, untouched

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

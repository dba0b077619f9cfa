"""The mixture-of-experts entry points on the GPU at the edges of what they allow: the largest and smallest
sizes of a launch, values at the ends of their types' range, empty plans, calls next to each other."""
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

"""The entry points of include/fp4q_experts.h: exported, typed, refusing bad
arguments on the host before anything is enqueued (no GPU needed: the fake
addresses are never dereferenced), and the row layout's arithmetic."""
import os
import re

import numpy as np
import pytest
import torch

import expert_ref as ref
import microscaling_fp4_quantization_bf16_b200 as fp4q
from microscaling_fp4_quantization_bf16_b200 import _abi, build, experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp4q_experts.h")

OK, NULL, SHAPE, ALIGN, UNSUP, ALIAS, CUDA = range(7)
A, A2, A3, A4, A5, A6 = (0x100000 * i for i in range(1, 7))
MIS = 0x100008   # 8-byte but not 16-byte aligned
ODD = 0x100002   # not 4-byte aligned
NV, MX, UE = 0, 1, 2
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"\b(fp4q_[a-z0-9_]+)\s*\(", text)))


def test_header_and_library_agree(lib):
    assert declared() == sorted(_abi.EXPERT_SIGNATURES)
    for n in declared():
        assert hasattr(lib, n)


def test_header_is_plain_c(tmp_path):
    import shutil
    import subprocess
    inc = "/usr/local/cuda/include"
    if shutil.which("gcc") is None or not os.path.exists(os.path.join(inc, "cuda_runtime_api.h")):
        pytest.skip("gcc or the CUDA headers are not available")
    for cc, std, name in (("gcc", "-std=c11", "h.c"), ("g++", "-std=c++17", "h.cpp")):
        f = tmp_path / name
        f.write_text('#include "fp4q_experts.h"\nint main(void) { return (int)FP4Q_ACT_SILU; }\n')
        r = subprocess.run([cc, std, "-Wall", "-Wextra", "-pedantic", "-Werror", "-I" + os.path.dirname(HEADER),
                            "-I" + inc, "-c", str(f), "-o", str(f) + ".o"], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("seed", range(20))
def test_rows_hold_every_routing(lib, seed):
    rng = np.random.default_rng(seed)
    n, e = int(rng.integers(0, 3000)), int(rng.integers(1, 300))
    rows = lib.fp4q_expert_rows(n, e)
    assert rows % 128 == 0
    worst = [np.arange(n) % e, np.zeros(n, int), rng.integers(0, e, n), np.minimum(np.arange(n), e - 1)]
    for ids in worst:
        assert ref.sort(ids[:, None], e)[1][-1] <= rows
    # and no fewer would do: one choice to each expert, the rest to one
    assert n == 0 or ref.sort(worst[3][:, None], e)[1][-1] > rows - 128 * 2


def test_rows_limits(lib):
    assert lib.fp4q_expert_rows(0, 8) == 0
    assert lib.fp4q_expert_rows(1, 1024) == 128
    for n, e in ((-1, 8), (4, 0), (4, 1025), (2 ** 31, 8), (2 ** 31 - 1, 1024)):
        assert lib.fp4q_expert_rows(n, e) == -1
        assert lib.fp4q_expert_sort_work(n, e) == -1
        with pytest.raises(ValueError):
            fp4q.expert_rows(n, e)
    # scratch: none while one block sorts, then a count per block and expert, at most 148 blocks
    assert lib.fp4q_expert_sort_work(1024, 64) == 0
    sizes = [lib.fp4q_expert_sort_work(n, 64) for n in (10 ** 4, 10 ** 5, 10 ** 6, 10 ** 8)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[-1] == 148 * 64 * 4


def test_sort_validation(lib):
    f = lambda ids=A, b=4, n=64, e=8, c=A2, s=A3, sl=A4, w=None: lib.fp4q_expert_sort(  # noqa: E731
        ids, b, n, e, c, s, sl, w, None)
    assert f(b=2) == UNSUP
    assert f(n=-1) == SHAPE
    assert f(e=0) == SHAPE
    assert f(e=1025) == SHAPE
    assert f(ids=None) == NULL
    assert f(c=None) == NULL
    assert f(s=None) == NULL
    assert f(sl=None) == NULL
    assert f(n=9000) == NULL                  # several blocks need work
    assert f(ids=ODD) == ALIGN
    assert f(b=8, ids=0x100004) == ALIGN
    assert f(c=ODD) == ALIGN
    assert f(n=9000, w=ODD) == ALIGN


def test_quantize_validation(lib):
    def f(x=A, tokens=4, cols=64, k=2, slots=A2, rows=256, fmt=NV, strat=0, rot=0, gin=A3, gout=A4, work=None,
          codes=A5, scales=A6, dq=None, dt=0):
        return lib.fp4q_expert_quantize(x, tokens, cols, k, slots, rows, fmt, strat, rot, gin, gout, work, codes,
                                        scales, dq, dt, None)
    assert f(fmt=UE) == UNSUP
    assert f(strat=4) == UNSUP
    assert f(fmt=MX, strat=2) == UNSUP
    assert f(rot=8) == UNSUP
    assert f(dq=A, dt=2) == UNSUP
    assert f(cols=48) == SHAPE
    assert f(cols=96, rot=64) == SHAPE
    assert f(rows=100) == SHAPE
    assert f(rows=-128) == SHAPE
    assert f(tokens=-1) == SHAPE
    assert f(k=0) == SHAPE
    assert f(k=65) == SHAPE
    assert f(tokens=2 ** 30, cols=256) == SHAPE   # 2^33 segments
    assert f(x=None) == NULL
    assert f(slots=None) == NULL
    assert f(codes=None) == NULL
    assert f(scales=None) == NULL
    assert f(gout=None) == NULL
    assert f(gin=None) == NULL                    # neither an abs-max nor scratch for one
    assert f(gin=A4) == ALIAS
    assert f(gin=None, work=A4) == ALIAS
    assert f(x=MIS) == ALIGN
    assert f(codes=MIS) == ALIGN
    assert f(scales=MIS) == ALIGN
    assert f(dq=MIS) == ALIGN
    assert f(slots=ODD) == ALIGN
    assert f(gout=ODD) == ALIGN


def test_product_validation(lib):
    def f(a=A, sa=A2, ga=A3, w=A4, sw=A5, gw=A6, c=A, s=A, e=4, rows=256, n=64, k=64, fmt=NV, mean=4, d=A2, dt=BF16):
        return lib.fp4q_expert_gemm(a, sa, ga, w, sw, gw, c, s, e, rows, n, k, fmt, mean, d, dt, None)
    assert f(fmt=UE) == UNSUP
    assert f(dt=2) == UNSUP
    assert f(k=48) == SHAPE
    assert f(k=0) == SHAPE
    assert f(n=12) == SHAPE
    assert f(n=6, dt=F32) == SHAPE
    assert f(rows=100) == SHAPE
    assert f(e=0) == SHAPE
    assert f(e=1025) == SHAPE
    assert f(mean=-1) == SHAPE
    assert f(e=1024, n=2 ** 24) == SHAPE
    for name in ("a", "sa", "ga", "w", "sw", "gw", "c", "s", "d"):
        assert f(**{name: None}) == NULL, name
    for name in ("a", "sa", "w", "sw", "d"):
        assert f(**{name: MIS}) == ALIGN, name
    for name in ("ga", "gw", "c", "s"):
        assert f(**{name: ODD}) == ALIGN, name
    assert f(rows=0, a=None) == OK                # nothing to do


def test_glu_validation(lib):
    def f(gu=A, rows=4, cols=64, slots=None, n=0, act=0, fmt=NV, strat=0, rot=0, gin=A3, gout=A4, work=None, codes=A5,
          scales=A6, dq=None, dt=0):
        return lib.fp4q_glu_quantize(gu, rows, cols, slots, n, act, fmt, strat, rot, gin, gout, work, codes, scales,
                                     dq, dt, None)
    assert f(act=2) == UNSUP
    assert f(fmt=UE) == UNSUP
    assert f(fmt=MX, strat=1) == UNSUP
    assert f(cols=40) == SHAPE
    assert f(rows=-1) == SHAPE
    assert f(slots=A2, n=-1) == SHAPE
    assert f(gu=None) == NULL
    assert f(codes=None) == NULL
    assert f(gin=None) == NULL
    assert f(gin=A4) == ALIAS
    assert f(gu=MIS) == ALIGN
    assert f(slots=ODD, n=4) == ALIGN
    b = lambda gu=A, dh=A2, rows=4, cols=64, act=0, rot=0, out=A3: lib.fp4q_glu_bwd(  # noqa: E731
        gu, dh, rows, cols, None, 0, act, rot, out, None)
    assert b(act=5) == UNSUP
    assert b(rot=24) == UNSUP
    assert b(cols=12) == SHAPE
    assert b(cols=48, rot=16) == SHAPE
    assert b(dh=None) == NULL
    assert b(out=MIS) == ALIGN
    assert b(rows=0, gu=None) == OK


def test_combine_validation(lib):
    def f(y=A, yt=BF16, rows=128, cols=64, slots=A2, tokens=4, k=2, w=None, rot=0, out=A3, ot=BF16):
        return lib.fp4q_expert_combine(y, yt, rows, cols, slots, tokens, k, w, rot, out, ot, None)
    assert f(yt=2) == UNSUP
    assert f(ot=7) == UNSUP
    assert f(rot=4) == UNSUP
    assert f(k=0) == SHAPE
    assert f(cols=12) == SHAPE
    assert f(cols=64, rot=128) == SHAPE
    assert f(y=None) == NULL
    assert f(slots=None) == NULL
    assert f(out=None) == NULL
    assert f(y=MIS) == ALIGN
    assert f(w=ODD) == ALIGN
    assert f(tokens=0, y=None) == OK

    def b(g=A, gt=BF16, y=A4, yt=BF16, rows=128, cols=64, slots=A2, tokens=4, k=2, w=None, dy=A3, dw=A5):
        return lib.fp4q_expert_combine_bwd(g, gt, y, yt, rows, cols, slots, tokens, k, w, dy, dw, None)
    assert b(gt=2) == UNSUP
    assert b(k=65) == SHAPE
    assert b(cols=4) == SHAPE
    assert b(y=None) == NULL                      # dweights need it
    assert b(dy=None) == NULL
    assert b(dw=ODD) == ALIGN
    assert b(tokens=0, g=None) == OK


def test_injected_cuda_error(lib):
    """Every entry point that enqueues work validates, then reports the injected error and touches nothing."""
    bufs = [np.full(1 << 16, 0xA5, np.uint8) for _ in range(9)]
    p = [b.ctypes.data for b in bufs]
    assert all(x % 16 == 0 for x in p)
    calls = {
        "fp4q_expert_sort": lambda: lib.fp4q_expert_sort(p[0], 4, 8, 2, p[1], p[2], p[3], None, None),
        "fp4q_expert_quantize": lambda: lib.fp4q_expert_quantize(p[0], 4, 64, 2, p[1], 128, NV, 0, 0, None, p[2], p[3],
                                                                 p[4], p[5], None, 0, None),
        "fp4q_expert_gemm": lambda: lib.fp4q_expert_gemm(*p[:8], 4, 128, 64, 64, NV, 1, p[8], BF16, None),
        "fp4q_glu_quantize": lambda: lib.fp4q_glu_quantize(p[0], 4, 64, None, 0, 0, NV, 0, 0, None, p[2], p[3], p[4],
                                                           p[5], None, 0, None),
        "fp4q_glu_bwd": lambda: lib.fp4q_glu_bwd(p[0], p[1], 4, 64, None, 0, 0, 0, p[2], None),
        "fp4q_expert_combine": lambda: lib.fp4q_expert_combine(p[0], BF16, 128, 64, p[1], 4, 2, None, 0, p[2], BF16,
                                                               None),
        "fp4q_expert_combine_bwd": lambda: lib.fp4q_expert_combine_bwd(p[0], BF16, p[1], BF16, 128, 64, p[2], 4, 2,
                                                                       None, p[3], p[4], None),
    }
    assert set(calls) == set(declared()) - {"fp4q_expert_rows", "fp4q_expert_sort_work"}
    try:
        for i, (name, call) in enumerate(calls.items()):
            lib.fp4q_debug_fail_launches(700 + i)
            assert call() == CUDA, name
            assert lib.fp4q_last_cuda_error() == 700 + i
    finally:
        lib.fp4q_debug_fail_launches(0)
    assert all((b == 0xA5).all() for b in bufs)


def test_python_refusals():
    """What the wrappers refuse before the library is called."""
    cpu = torch.zeros(4, 2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        fp4q.expert_sort(cpu, 4)
    plan = fp4q.ExpertPlan(torch.zeros(4), torch.zeros(5), torch.zeros(4, 2), 128)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: fp4q.expert_quantize(x, plan), lambda: fp4q.glu_quantize(x), lambda: fp4q.glu_bwd(x, x),
                 lambda: fp4q.expert_combine(x, plan), lambda: fp4q.expert_combine_bwd(x, x, plan),
                 lambda: fp4q.expert_weights(x), lambda: fp4q.expert_gemm(x, x, x, x, x, x, plan)):
        with pytest.raises(ValueError):
            call()
    for fmt in ("ue5m3", "int4", 2, None):
        with pytest.raises(ValueError):
            experts._fmt(fmt)
    with pytest.raises(ValueError):
        experts._strategy("best")
    with pytest.raises(ValueError):
        experts._act("relu")


def test_scale_bytes_agree(lib):
    for fmt, f in (("nvfp4", NV), ("mxfp4", MX)):
        for rows, cols in ((1, 32), (128, 64), (300, 1056), (5, 4096)):
            assert experts.scale_bytes(rows, cols, fmt) == lib.fp4q_mma_scale_bytes(rows, cols, f)


@pytest.mark.parametrize("strategy", ["absmax", "prevent_zero", "four_over_six", "brute_force"])
@pytest.mark.parametrize("rot", [0, 16, 128])
def test_reference_steps_are_the_oracles(strategy, rot):
    """The fp32 steps that the GPU tests hold NVFP4 without a given abs-max to, against the oracle under its s_g."""
    rng = np.random.default_rng(rot)
    x = torch.from_numpy(rng.laplace(0, 1, (24, 256)) * (1 + 20 * (rng.random((24, 256)) < 0.01))).to(torch.bfloat16)
    x[3, :64] = 0
    x[4] *= 2.0 ** -40
    bits = ref.bits(x)
    want = ref.quantize(bits, "nvfp4", strategy, rot, 77.0)
    y = ref._rotate32((bits.astype(np.uint32) << 16).view(np.float32), rot)
    got = ref._nvfp4(y, strategy, np.float32(77.0) / np.float32(2688))
    for k in ("codes", "scales", "dq"):
        assert np.array_equal(got[k], want[k]), k

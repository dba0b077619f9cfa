"""One mixture-of-experts feed-forward layer in FP4: the torch side of
include/fp4q_experts.h.

    plan = expert_sort(ids, experts)                        # rows of the expert order
    qa = expert_quantize(x, plan, "nvfp4")                  # tokens -> quantized rows
    gu = expert_gemm(qa.codes, qa.scales, qa.global_scale, up.codes, up.scales,
                     up.global_scale, plan, "nvfp4")        # gate and value of every row
    qh = glu_quantize(gu, "nvfp4", plan=plan)               # silu(gate) * value, quantized
    y = expert_gemm(qh.codes, qh.scales, qh.global_scale, down.codes, down.scales,
                    down.global_scale, plan, "nvfp4")
    out = expert_combine(y, plan, weights)                  # weighted sum back to tokens

The weights are laid out once by expert_weights(). Every function runs on the
current stream of its tensors' device and allocates its outputs with torch
(unless given preallocated ones); nothing reads a size back from the device,
so a whole layer can be captured in a CUDA graph. Rows of the padded layout
that hold no choice are left as they were.
"""
from __future__ import annotations

import functools
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import _abi

ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}
SEGMENT_ROWS = 128
AMAX_WORK = 1024
_FORMATS = {"nvfp4": 0, "mxfp4": 1}
_STRATEGIES = {"absmax": 0, "prevent_zero": 1, "four_over_six": 2, "brute_force": 3}
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}


@dataclass
class ExpertPlan:
    """Where each choice's row is (see include/fp4q_experts.h)."""
    counts: torch.Tensor   # int32 [experts]: choices of each expert
    starts: torch.Tensor   # int32 [experts + 1]: first row of each, a multiple of 128
    slots: torch.Tensor    # int32 [tokens, k]: row of each choice, -1 if dropped
    rows: int              # rows of the padded layout, a multiple of 128


@dataclass
class ExpertWeights:
    """One weight matrix per expert in the product's operand form."""
    codes: torch.Tensor                   # uint8 [experts, N, K/2]
    scales: torch.Tensor                  # uint8 [experts, mma_scale_bytes(N, K)]
    global_scale: Optional[torch.Tensor]  # float32 [experts] (NVFP4) or None


def _need(t, name: str, device, dtype, *shape) -> None:
    """t is a contiguous tensor on `device` of dtype (or one of several) and shape (None: any)."""
    try:
        if (t.device == device and (t.dtype is dtype or t.dtype in dtype) and t.is_contiguous()
                and (not shape or t.shape == shape)):
            return
    except (AttributeError, TypeError):
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"all tensors must be on {device}, {name} is on {t.device}")
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape and (t.dim() != len(shape) or any(s is not None and s != d
                                               for s, d in zip(shape, t.shape))):
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


def _device(t, name: str) -> torch.device:
    """The CUDA device of a call's first tensor, which all the others must share."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _matrix(t, name: str, device, dtype):
    """The shape of t, a contiguous matrix on `device` of dtype (or one of several)."""
    _need(t, name, device, dtype)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(shape)}")
    return shape


def _result(dtype, name: str):
    """dtype, if results can have it."""
    if dtype not in _DTYPES:
        raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, got {dtype}")
    return dtype


def _fmt(fmt) -> int:
    f = _FORMATS.get(fmt) if isinstance(fmt, str) else fmt
    if f not in (0, 1):
        raise ValueError(f"fmt must be 'nvfp4' or 'mxfp4', got {fmt!r}")
    return f


def _strategy(s) -> int:
    v = _STRATEGIES.get(s) if isinstance(s, str) else s
    if v not in (0, 1, 2, 3):
        raise ValueError(f"unknown strategy {s!r}")
    return v


def _act(act) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    return ACTIVATIONS[act]


_bound = {}  # entry points of the loaded library, by name


def _entry(name: str):
    fn = _bound.get(name)
    if fn is None:
        fn = _bound[name] = getattr(_abi.load(), name)
    return fn


def _call(name: str, device: torch.device, *args) -> None:
    """Calls an entry point on the current stream of `device`."""
    index = device.index
    if index == torch._C._cuda_getDevice():
        status = _entry(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = _entry(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _abi.fail(name, status)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _plan_args(plan: ExpertPlan, device) -> None:
    _matrix(plan.slots, "plan.slots", device, torch.int32)
    if plan.rows < 0 or plan.rows % SEGMENT_ROWS:
        raise ValueError(f"plan.rows must be a multiple of {SEGMENT_ROWS}, got {plan.rows}")


def _rows_taken(plan: Optional[ExpertPlan], rows: int, device):
    """(rows, slots, their number) of a call over a plan's rows of a [rows, ...] input, over all without one.
    To the library no slots means all rows, and an empty tensor's address is none: a plan without a choice
    takes no row, so its call has none."""
    if plan is None:
        return rows, None, rows
    _plan_args(plan, device)
    if plan.rows != rows:
        raise ValueError(f"gu has {rows} rows, the plan {plan.rows}")
    n = plan.slots.numel()
    return (rows, plan.slots.data_ptr(), n) if n else (0, None, 0)


@functools.lru_cache(maxsize=4096)
def scale_bytes(rows: int, cols: int, fmt="nvfp4") -> int:
    """Bytes of the MMA-layout scales of [rows, cols] (0 rows or columns: 0)."""
    blocks = cols // (16 if _fmt(fmt) == 0 else 32)
    return -(-rows // 128) * 128 * (-(-blocks // 4) * 4)


@functools.lru_cache(maxsize=4096)
def expert_rows(choices: int, experts: int) -> int:
    """Rows of the padded layout that hold any routing of `choices` choices."""
    rows = _entry("fp4q_expert_rows")(choices, experts)
    if rows < 0:
        raise ValueError(f"no row layout for {choices} choices among {experts} experts")
    return rows


@functools.lru_cache(maxsize=4096)
def _sort_work(choices: int, experts: int) -> int:
    return _entry("fp4q_expert_sort_work")(choices, experts)


def expert_sort(ids: torch.Tensor, experts: int, rows: Optional[int] = None,
                out: Optional[ExpertPlan] = None) -> ExpertPlan:
    """Sorts the router's choices ids (int32 or int64 [tokens, k]) by expert,
    stably. An id outside 0 .. experts-1 drops the choice. rows: rows of the
    layout, at least the default expert_rows(tokens * k, experts)."""
    dev = _device(ids, "ids")
    _matrix(ids, "ids", dev, (torch.int32, torch.int64))
    n = ids.numel()
    least = expert_rows(n, experts)
    if out is None:
        out = ExpertPlan(torch.empty(experts, dtype=torch.int32, device=dev),
                         torch.empty(experts + 1, dtype=torch.int32, device=dev),
                         torch.empty(ids.shape, dtype=torch.int32, device=dev),
                         least if rows is None else rows)
    else:
        _need(out.counts, "out.counts", dev, torch.int32, experts)
        _need(out.starts, "out.starts", dev, torch.int32, experts + 1)
        _need(out.slots, "out.slots", dev, torch.int32, *ids.shape)
    if out.rows < least or out.rows % SEGMENT_ROWS:
        raise ValueError(f"rows must be a multiple of {SEGMENT_ROWS} and at least {least}, got {out.rows}")
    size = _sort_work(n, experts)
    work = torch.empty(size // 4, dtype=torch.int32, device=dev) if size else None
    _call("fp4q_expert_sort", dev, ids.data_ptr(), ids.element_size(), n, experts,
          out.counts.data_ptr(), out.starts.data_ptr(), out.slots.data_ptr(), _ptr(work))
    return out


def _quantized_out(out, rows: int, cols: int, f: int, dq_dtype, device):
    """The given Quantized, checked, or a new one for [rows, cols] in the MMA layout."""
    from . import Quantized
    size = scale_bytes(rows, cols, f)
    if out is None:
        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=device)
        return Quantized(new((rows, cols // 2), torch.uint8), new((size,), torch.uint8),
                         new((1,), torch.float32) if f == 0 else None, None,
                         new((rows, cols), _result(dq_dtype, "dq_dtype")) if dq_dtype is not None else None)
    _need(out.codes, "out.codes", device, torch.uint8, rows, cols // 2)
    _need(out.scales, "out.scales", device, torch.uint8, size)
    if f == 0:
        _need(out.global_scale, "out.global_scale", device, torch.float32, 1)
    if out.dq is not None:
        _need(out.dq, "out.dq", device, (torch.float32, torch.bfloat16), rows, cols)
    return out


def _amax_args(f: int, global_amax, device):
    """(calibrated abs-max or None, scratch for a computed one or None)."""
    if f != 0:
        return None, None
    if global_amax is not None:
        _need(global_amax, "global_amax", device, torch.float32, 1)
        return global_amax, None
    return None, torch.empty(AMAX_WORK, dtype=torch.float32, device=device)


def expert_quantize(x: torch.Tensor, plan: ExpertPlan, fmt="nvfp4", strategy="absmax", rot: int = 0,
                    global_amax: Optional[torch.Tensor] = None,
                    dq_dtype: Optional[torch.dtype] = None, out=None):
    """quantize_mma() of bf16 tokens [tokens, cols] into the rows of their
    choices; each token is quantized once. Returns a Quantized of
    [plan.rows, cols] with MMA-layout scales (and dequantized values in
    .dq, if dq_dtype or out.dq asks for them). NVFP4 without global_amax takes the
    abs-max of x in an extra pass (see fp4q_expert_quantize for its s_g)."""
    dev = _device(x, "x")
    tokens, cols = _matrix(x, "x", dev, torch.bfloat16)
    _plan_args(plan, dev)
    if plan.slots.shape[0] != tokens:
        raise ValueError(f"x has {tokens} tokens, the plan {plan.slots.shape[0]}")
    f = _fmt(fmt)
    out = _quantized_out(out, plan.rows, cols, f, dq_dtype, dev)
    amax, work = _amax_args(f, global_amax, dev)
    _call("fp4q_expert_quantize", dev, x.data_ptr(), tokens, cols, plan.slots.shape[1],
          plan.slots.data_ptr(), plan.rows, f, _strategy(strategy), rot, _ptr(amax),
          _ptr(out.global_scale) if f == 0 else None, _ptr(work), out.codes.data_ptr(),
          out.scales.data_ptr(), _ptr(out.dq), _DTYPES[out.dq.dtype] if out.dq is not None else 0)
    return out


def expert_weights(w: torch.Tensor, fmt="nvfp4", strategy="absmax", rot: int = 0) -> ExpertWeights:
    """Quantizes bf16 weights [experts, N, K] for expert_gemm, each expert with
    its own scales (done once, when a model is loaded)."""
    from . import Quantized, quantize_mma
    dev = _device(w, "w")
    _need(w, "w", dev, torch.bfloat16)
    if w.dim() != 3:
        raise ValueError(f"w must have shape [experts, N, K], got {tuple(w.shape)}")
    experts, n, k = w.shape
    f = _fmt(fmt)
    out = ExpertWeights(
        torch.empty(experts, n, k // 2, dtype=torch.uint8, device=dev),
        torch.zeros(experts, scale_bytes(n, k, f), dtype=torch.uint8, device=dev),
        torch.empty(experts, dtype=torch.float32, device=dev) if f == 0 else None)
    with torch.cuda.device(dev):
        for e in range(experts):
            gs = out.global_scale[e:e + 1] if f == 0 else None
            quantize_mma(w[e], fmt, strategy, rot,
                         out=Quantized(out.codes[e], out.scales[e], gs, None, None))
    return out


def expert_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, a_global_scale: Optional[torch.Tensor],
                w_codes: torch.Tensor, w_scales: torch.Tensor, w_global_scale: Optional[torch.Tensor],
                plan: ExpertPlan, fmt="nvfp4", out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Each row times its expert's weights, W4A4: [rows, K] x [experts, N, K]
    -> [rows, N]. Operands as expert_quantize / glu_quantize and expert_weights
    return them."""
    f = _fmt(fmt)
    dev = _device(w_codes, "w_codes")
    _need(w_codes, "w_codes", dev, torch.uint8)
    if w_codes.dim() != 3 or w_codes.shape[0] == 0:
        raise ValueError(f"w_codes must have shape [experts, N, K/2], got {tuple(w_codes.shape)}")
    experts, n, half = w_codes.shape
    k = 2 * half
    _plan_args(plan, dev)
    rows = plan.rows
    _need(a_codes, "a_codes", dev, torch.uint8, rows, half)
    _need(a_scales, "a_scales", dev, torch.uint8, scale_bytes(rows, k, f))
    _need(w_scales, "w_scales", dev, torch.uint8, experts, scale_bytes(n, k, f))
    _need(plan.counts, "plan.counts", dev, torch.int32, experts)
    _need(plan.starts, "plan.starts", dev, torch.int32, experts + 1)
    if f == 0:
        _need(a_global_scale, "a_global_scale", dev, torch.float32, 1)
        _need(w_global_scale, "w_global_scale", dev, torch.float32, experts)
    else:
        a_global_scale = w_global_scale = None
    if out is None:
        out = torch.empty(rows, n, dtype=_result(out_dtype, "out_dtype"), device=dev)
    else:
        _need(out, "out", dev, (torch.float32, torch.bfloat16), rows, n)
    choices = plan.slots.numel()
    _call("fp4q_expert_gemm", dev, a_codes.data_ptr(), a_scales.data_ptr(), _ptr(a_global_scale),
          w_codes.data_ptr(), w_scales.data_ptr(), _ptr(w_global_scale), plan.counts.data_ptr(),
          plan.starts.data_ptr(), experts, rows, n, k, f, -(-choices // experts), out.data_ptr(),
          _DTYPES[out.dtype])
    return out


def glu_quantize(gu: torch.Tensor, fmt="nvfp4", strategy="absmax", rot: int = 0,
                 plan: Optional[ExpertPlan] = None, act: str = "silu",
                 global_amax: Optional[torch.Tensor] = None,
                 dq_dtype: Optional[torch.dtype] = None, out=None):
    """Gated activation and quantize_mma() in one pass: gu bf16 [rows, 2 * cols]
    (gate, then value) -> Quantized of act(gate) * value. With a plan only the
    rows that hold a choice are taken, without one all rows."""
    dev = _device(gu, "gu")
    rows, cols = _matrix(gu, "gu", dev, torch.bfloat16)
    cols, odd = cols // 2, cols % 2
    if odd:
        raise ValueError("gu must have an even number of columns")
    taken, slots, n = _rows_taken(plan, rows, dev)
    f = _fmt(fmt)
    out = _quantized_out(out, rows, cols, f, dq_dtype, dev)
    amax, work = _amax_args(f, global_amax, dev)
    _call("fp4q_glu_quantize", dev, gu.data_ptr(), taken, cols, slots, n, _act(act), f, _strategy(strategy), rot,
          _ptr(amax), _ptr(out.global_scale) if f == 0 else None, _ptr(work), out.codes.data_ptr(),
          out.scales.data_ptr(), _ptr(out.dq), _DTYPES[out.dq.dtype] if out.dq is not None else 0)
    return out


def glu_bwd(gu: torch.Tensor, dh: torch.Tensor, plan: Optional[ExpertPlan] = None, act: str = "silu",
            rot: int = 0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of glu_quantize's gate and value (bf16 [rows, 2 * cols]) from
    dh = dL/d(quantized values) bf16 [rows, cols], straight through the rounding."""
    dev = _device(gu, "gu")
    rows, cols = _matrix(gu, "gu", dev, torch.bfloat16)
    cols, odd = cols // 2, cols % 2
    _need(dh, "dh", dev, torch.bfloat16, rows, cols)
    if odd:
        raise ValueError("gu must have an even number of columns")
    taken, slots, n = _rows_taken(plan, rows, dev)
    if out is None:
        out = torch.empty_like(gu)
    else:
        _need(out, "out", dev, torch.bfloat16, rows, 2 * cols)
    _call("fp4q_glu_bwd", dev, gu.data_ptr(), dh.data_ptr(), taken, cols, slots, n, _act(act), rot,
          out.data_ptr())
    return out


def expert_combine(y: torch.Tensor, plan: ExpertPlan, weights: Optional[torch.Tensor] = None,
                   rot: int = 0, out_dtype: torch.dtype = torch.bfloat16,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[slots[t, j]] (weights None: ones), then
    the rotation. Without weights and with the forward's rot it is the
    straight-through gradient of expert_quantize."""
    dev = _device(y, "y")
    rows, cols = _matrix(y, "y", dev, (torch.float32, torch.bfloat16))
    _plan_args(plan, dev)
    if rows != plan.rows:
        raise ValueError(f"y has {rows} rows, the plan {plan.rows}")
    tokens, k = plan.slots.shape
    if weights is not None:
        _need(weights, "weights", dev, torch.float32, tokens, k)
    if out is None:
        out = torch.empty(tokens, cols, dtype=_result(out_dtype, "out_dtype"), device=dev)
    else:
        _need(out, "out", dev, (torch.float32, torch.bfloat16), tokens, cols)
    _call("fp4q_expert_combine", dev, y.data_ptr(), _DTYPES[y.dtype], plan.rows, cols,
          plan.slots.data_ptr(), tokens, k, _ptr(weights), rot, out.data_ptr(), _DTYPES[out.dtype])
    return out


def expert_combine_bwd(g: torch.Tensor, y: torch.Tensor, plan: ExpertPlan,
                       weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       want_dweights: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradients of expert_combine (rot 0) from g = dL/dout: (dy of y's type
    and shape, dweights float32 [tokens, k] or None)."""
    dev = _device(y, "y")
    rows, cols = _matrix(y, "y", dev, (torch.float32, torch.bfloat16))
    _plan_args(plan, dev)
    if rows != plan.rows:
        raise ValueError(f"y has {rows} rows, the plan {plan.rows}")
    tokens, k = plan.slots.shape
    _need(g, "g", dev, (torch.float32, torch.bfloat16), tokens, cols)
    if weights is not None:
        _need(weights, "weights", dev, torch.float32, tokens, k)
    if out is None:
        out = torch.empty_like(y)
    else:
        _need(out, "out", dev, y.dtype, plan.rows, cols)
    dw = torch.empty(tokens, k, dtype=torch.float32, device=dev) if want_dweights else None
    if dw is not None and cols == 0:
        dw.zero_()
    _call("fp4q_expert_combine_bwd", dev, g.data_ptr(), _DTYPES[g.dtype], y.data_ptr(),
          _DTYPES[y.dtype], plan.rows, cols, plan.slots.data_ptr(), tokens, k, _ptr(weights),
          out.data_ptr(), _ptr(dw))
    return out, dw

"""The operators of one mixture-of-experts feed-forward layer in FP4, as cases that can be timed and compared.

Five operators: tokens sorted by expert, their quantization in expert order, the grouped W4A4 product, the gated
activation in front of the second product (with its gradient), and the weighted sum back to tokens (with its gradient).
Where ``own`` is false, ``run`` computes them with elementary torch operations; where it is true, through this
repository's package.

The quantizer's definition is one binary32 operation per step (butterflies in ascending order, u = y * fl(1 / S), block
sums by the adjacent-pair tree), so the plain forms take the same steps; the activation is taken in 64 bits, because its
rounding to bf16 decides codes.
"""
import math

import torch

own = False

PAD = 128        # rows of the padded layout: every expert's segment starts at a multiple of this
DROP = 0.03      # share of choices that are dropped, where a case has dropped choices

_E2M1_STEPS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)    # midpoints between neighbouring E2M1 magnitudes
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
_BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the router's choices of a small batch at decode time: a launch's latency
        {"name": "sort, 64 tokens", "op": "sort", "tokens": 64, "k": 2, "experts": 8, "wide": True, "drop": False},
        # a training or prefill step with many small experts, some choices dropped by capacity
        {"name": "sort, 65536 tokens", "op": "sort", "tokens": 65536, "k": 8, "experts": 256, "wide": False, "drop": True},
        # activations of a decode batch in front of the up projections
        {"name": "quantize, 33 tokens mxfp4", "op": "quantize", "tokens": 33, "k": 4, "experts": 32, "cols": 4096, "fmt": "mxfp4",
         "strategy": "absmax", "rot": 32, "calibrated": True, "drop": False},
        # activations of a prefill batch at this repository's largest activation shape, two experts a token
        {"name": "quantize, 16384 tokens nvfp4", "op": "quantize", "tokens": 16384, "k": 2, "experts": 16, "cols": 8192, "fmt": "nvfp4",
         "strategy": "four_over_six", "rot": 16, "calibrated": True, "drop": True},
        # decode: few rows for each expert, bound by reading the weights
        {"name": "gemm, 32 tokens nvfp4", "op": "gemm", "tokens": 32, "k": 4, "experts": 32, "cols": 4096, "outs": 4096, "fmt": "nvfp4",
         "f32": False, "drop": False},
        # prefill: few large experts, bound by the tensor cores
        {"name": "gemm, 8192 tokens nvfp4", "op": "gemm", "tokens": 8192, "k": 2, "experts": 8, "cols": 4096, "outs": 14336, "fmt": "nvfp4",
         "f32": False, "drop": False},
        # odd sizes, ragged segments, dropped choices, 32-bit results
        {"name": "gemm, 1000 tokens mxfp4 f32", "op": "gemm", "tokens": 1000, "k": 3, "experts": 12, "cols": 1056, "outs": 1412, "fmt": "mxfp4",
         "f32": True, "drop": True},
        # the activation between the two products of a decode batch, global scale from the rows themselves
        {"name": "glu, 48 tokens nvfp4", "op": "glu", "tokens": 48, "k": 1, "experts": 8, "inner": 2048, "fmt": "nvfp4",
         "strategy": "absmax", "rot": 0, "act": "silu", "calibrated": False, "drop": False},
        # and of a prefill batch, wide inner size
        {"name": "glu, 8192 tokens mxfp4", "op": "glu", "tokens": 4096, "k": 2, "experts": 8, "inner": 14336, "fmt": "mxfp4",
         "strategy": "absmax", "rot": 128, "act": "silu", "calibrated": True, "drop": True},
        # its gradient in a calibration step
        {"name": "glu gradient, 6001 tokens", "op": "glu_bwd", "tokens": 6001, "k": 1, "experts": 16, "inner": 4096, "rot": 16,
         "act": "gelu_tanh", "drop": True},
        # expert outputs back to tokens after a prefill, eight experts a token
        {"name": "combine, 8192 tokens", "op": "combine", "tokens": 8192, "k": 8, "experts": 64, "cols": 4096, "weighted": True,
         "rot": 0, "f32": False, "drop": True},
        # its gradient, for the expert outputs and the router's weights
        {"name": "combine gradient, 4000 tokens", "op": "combine_bwd", "tokens": 4000, "k": 4, "experts": 32, "cols": 4096,
         "drop": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("sort", "quantize", "gemm", "gemm", "glu", "glu_bwd", "combine", "combine_bwd"))
    experts = rng.choice((4, 7, 8, 16, 24, 32, 60, 64, 128, 256))
    k = rng.randint(1, min(8, experts))
    case = {"op": op, "k": k, "experts": experts, "drop": rng.random() < 0.5}
    fmt = rng.choice(("nvfp4", "mxfp4"))
    rot = rng.choice((0, 0, 16, 32, 64, 128))
    width = 128 * _log(rng, 2, 64) if rot else 32 * _log(rng, 4, 256)
    strategy = rng.choice(("absmax", "prevent_zero", "four_over_six")) if fmt == "nvfp4" else "absmax"
    quant = {"fmt": fmt, "strategy": strategy, "rot": rot, "calibrated": rng.random() < 0.6}
    if op == "sort":
        return dict(case, tokens=_log(rng, 1, 500000 / k), wide=rng.random() < 0.5)
    if op == "quantize":
        return dict(case, tokens=_log(rng, 1, min(16384, 2.6e8 / (width * k))), cols=width, **quant)
    if op == "gemm":
        cols = 32 * _log(rng, 4, 224)
        outs = 8 * _log(rng, 8, 1024)
        experts = max(1, min(experts, int(4.6e8 / (cols * outs))))
        k = min(k, experts)
        return dict(case, k=k, experts=experts, tokens=_log(rng, 1, min(8192, 9e11 / (2.0 * cols * outs * k))), cols=cols, outs=outs,
                    fmt=fmt, f32=rng.random() < 0.4)
    if op == "glu":
        return dict(case, tokens=_log(rng, 1, min(8192, 1.1e8 / (width * k))), inner=width, act=rng.choice(("silu", "gelu_tanh")), **quant)
    if op == "glu_bwd":
        return dict(case, tokens=_log(rng, 1, min(8192, 1.1e8 / (width * k))), inner=width, rot=rot, act=rng.choice(("silu", "gelu_tanh")))
    if op == "combine":
        weighted = rng.random() < 0.6
        return dict(case, tokens=_log(rng, 1, min(16384, 2.6e8 / (width * k))), cols=width, weighted=weighted, rot=0 if weighted else rot,
                    f32=rng.random() < 0.3)
    return dict(case, tokens=_log(rng, 1, min(16384, 1.3e8 / (width * k))), cols=width)


# ------------------------------------------------------------------------------------------------ inputs

def _rows(n, experts):
    """Rows of the padded layout that n routed choices can need at most."""
    return (n + (PAD - 1) * min(experts, n)) // PAD * PAD


def _route(case, g):
    """The router's choices int64 [tokens, k]: distinct experts of uneven popularity; -1 where a choice is dropped."""
    t, k, e = case["tokens"], case["k"], case["experts"]
    score = torch.randn(t, e, generator=g, device="cuda") + 0.7 * torch.randn(e, generator=g, device="cuda")
    ids = score.topk(k, dim=1).indices
    if case["drop"]:
        ids = torch.where(torch.rand(t, k, generator=g, device="cuda") < DROP, -1, ids)
    return ids


def _plan(ids, experts):
    """counts [E], starts [E + 1] and slots [T, k] of the padded layout: every expert's rows in token order."""
    flat = ids.reshape(-1)
    n = flat.numel()
    valid = (flat >= 0) & (flat < experts)
    key = torch.where(valid, flat, experts).long()
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(n, device=ids.device)
    first = counts.cumsum(0) - counts
    padded = (counts[:experts] + PAD - 1) // PAD * PAD
    starts = torch.cat((padded.new_zeros(1), padded.cumsum(0)))
    slots = torch.where(valid, starts[key] + place - first[key], -1)
    return counts[:experts].int(), starts.int(), slots.int().reshape(ids.shape)


def _activations(g, rows, cols):
    """bf16 activations: Laplace-like values with 1% of the channels twenty times larger."""
    u = torch.rand(rows, cols, generator=g, device="cuda") - 0.5
    x = -torch.sign(u) * torch.log1p(-2.0 * u.abs().clamp_(max=0.4999999))
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(torch.bfloat16)


def _normal(g, *shape, std=1.0):
    return (std * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = _route(case, g)
    op, n, experts = case["op"], case["tokens"] * case["k"], case["experts"]
    if op == "sort":
        return {"case": case, "ids": ids if case["wide"] else ids.int()}
    counts, starts, slots = _plan(ids, experts)
    rows = _rows(n, experts)
    s = {"case": case, "counts": counts, "starts": starts, "slots": slots, "rows": rows}
    fmt = case.get("fmt")
    if op == "quantize":
        s["x"] = _activations(g, case["tokens"], case["cols"])
        width = case["cols"]
    if op in ("glu", "glu_bwd"):
        s["gu"] = _normal(g, rows, 2 * case["inner"])
        width = case["inner"]
        if op == "glu_bwd":
            s["dh"] = _normal(g, rows, width)
            s["out"] = torch.zeros(rows, 2 * width, dtype=torch.bfloat16, device="cuda")
    if op in ("quantize", "glu"):
        # a calibrated abs-max covers the rotated values seen in calibration; the buffers are the program's own
        s["amax"] = torch.full((1,), 320.0 if op == "quantize" else 32.0, device="cuda") if case["calibrated"] and fmt == "nvfp4" else None
        s["codes"] = torch.zeros(rows, width // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(rows * _pad4(width // _BLOCK[fmt]), dtype=torch.uint8, device="cuda")
        s["global_scale"] = torch.zeros(1, device="cuda") if fmt == "nvfp4" else None
        s["dq"] = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    if op == "gemm":
        cols, outs = case["cols"], case["outs"]
        s["cap"] = int(counts.max()) if n else 0
        x = _activations(g, rows, cols)
        s["a"] = _operand(x[None], fmt)
        s["w"] = _operand(torch.stack([_normal(g, outs, cols, std=0.02) for _ in range(experts)]), fmt)
        s["out"] = torch.zeros(rows, outs, dtype=torch.float32 if case["f32"] else torch.bfloat16, device="cuda")
    if op in ("combine", "combine_bwd"):
        cols = case["cols"]
        s["y"] = _normal(g, rows, cols)
        w = torch.rand(case["tokens"], case["k"], generator=g, device="cuda") + 0.05
        s["weights"] = w / w.sum(1, keepdim=True) if case.get("weighted", True) else None
        if op == "combine_bwd":
            s["g"] = _normal(g, case["tokens"], cols)
            s["out"] = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _pad4(blocks):
    return -(-blocks // 4) * 4


def _pairs(x, n):
    """Adjacent-pair tree sum over the last axis of n values."""
    while n > 1:
        x = x[..., 0::2] + x[..., 1::2]
        n //= 2
    return x[..., 0]


def _rotate(y, rot):
    """Blockwise Walsh-Hadamard transform in 32 bits: butterflies of ascending distance, then one factor."""
    if not rot:
        return y
    shape, h = y.shape, 1
    while h < rot:
        p = y.reshape(-1, 2, h)
        y = torch.stack((p[:, 0] + p[:, 1], p[:, 0] - p[:, 1]), 1)
        h *= 2
    return y.reshape(shape) * torch.tensor(rot ** -0.5, dtype=torch.float32, device=y.device)


def _e2m1(u):
    """E2M1 index of each value, ties to the even one, the sign in bit 3."""
    a = u.abs()
    m = torch.zeros_like(a, dtype=torch.uint8)
    m += a > _E2M1_STEPS[0]
    m += a >= _E2M1_STEPS[1]
    m += a > _E2M1_STEPS[2]
    m += a >= _E2M1_STEPS[3]
    m += a > _E2M1_STEPS[4]
    m += a >= _E2M1_STEPS[5]
    m += a > _E2M1_STEPS[6]
    return m + 8 * torch.signbit(u).to(torch.uint8)


def _value(code):
    return torch.tensor(_E2M1, dtype=torch.float32, device=code.device)[code.int()]


def _encode(y, scale):
    """Codes of blocks y [..., B] under scale [..., 1], and the values that they stand for."""
    r = torch.where(scale == 0, 0.0, 1.0 / scale)
    code = torch.where(scale == 0, 0, _e2m1(y * r.clamp(max=torch.finfo(torch.float32).max)))
    return code, _value(code) * scale


def _blocks(y, fmt, strategy, amax):
    """(code, scale byte, values, global scale) of [..., cols] in blocks; amax: the tensor's abs-max (nvfp4)."""
    b = _BLOCK[fmt]
    y = y.reshape(*y.shape[:-1], -1, b)
    top = y.abs().amax(-1, keepdim=True)
    if fmt == "mxfp4":
        e = torch.where(top == 0, -127, torch.frexp(top).exponent - 3).clamp(-127, 127)
        scale = torch.ldexp(torch.ones_like(top), e)
        code, v = _encode(y, scale)
        return code, (e + 127).to(torch.uint8), v, None
    sg = amax / 2688.0
    sg = torch.where((sg > 0) & torch.isfinite(sg), sg, 1.0)

    def at(target):
        byte = (top / (sg * target)).clamp(max=448.0).to(torch.float8_e4m3fn)
        if strategy == "prevent_zero":
            byte = byte.view(torch.uint8).clamp(min=1).view(torch.float8_e4m3fn)
        scale = byte.float() * sg
        return (byte.view(torch.uint8),) + _encode(y, scale)

    byte, code, v = at(6.0)
    if strategy == "four_over_six":
        byte4, code4, v4 = at(4.0)
        d, d4 = y - v, y - v4
        four = (_pairs(d4 * d4, b) < _pairs(d * d, b))[..., None]
        byte, code, v = torch.where(four, byte4, byte), torch.where(four, code4, code), torch.where(four, v4, v)
    return code, byte, v, sg


def _mma_layout(byte):
    """Row-major scale bytes [R, blocks] -> 512-byte atoms of 128 rows x 4 blocks, atoms along the row first; padding is zero."""
    rows, blocks = byte.shape
    full = byte.new_zeros(-(-rows // PAD) * PAD, _pad4(blocks))
    full[:rows, :blocks] = byte
    return full.reshape(-1, 4, 32, full.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _row_major(flat, rows, blocks):
    """The way back from _mma_layout."""
    a = flat.reshape(-1, _pad4(blocks) // 4, 32, 4, 4).permute(0, 3, 2, 1, 4)
    return a.reshape(-1, _pad4(blocks))[:rows, :blocks]


def _operand(x, fmt):
    """Quantized operand of a product: packed codes, MMA-layout scales and global scales of bf16 [parts, rows, cols]."""
    parts, rows, cols = x.shape
    codes, scales, sgs = [], [], []
    for part in x:
        y = part.float()
        code, byte, _, sg = _blocks(y, fmt, "absmax", y.abs().amax())
        code = code.reshape(rows, cols)
        codes.append(code[:, 0::2] | (code[:, 1::2] << 4))
        scales.append(_mma_layout(byte.reshape(rows, -1)))
        sgs.append(sg)
    return torch.stack(codes), torch.stack(scales), torch.stack(sgs) if fmt == "nvfp4" else None


def _dequantized(operand, fmt, cols, dtype):
    """Values [parts, rows, cols] of an operand without its global scales."""
    codes, scales, _ = operand
    parts, rows = codes.shape[:2]
    b = _BLOCK[fmt]
    code = torch.stack((codes & 15, codes >> 4), -1).reshape(parts, rows, cols // b, b)
    byte = _row_major(scales, parts * -(-rows // PAD) * PAD, cols // b).reshape(parts, -1, cols // b)[:, :rows]
    if fmt == "nvfp4":
        scale = byte.contiguous().view(torch.float8_e4m3fn).to(dtype)
    else:
        scale = torch.ldexp(torch.ones_like(byte, dtype=dtype), byte.int() - 127)
    return (torch.tensor(_E2M1, dtype=dtype, device=code.device)[code.int()] * scale[..., None]).reshape(parts, rows, cols)


def _choice_of(s):
    """For every row of the padded layout the flat choice in it, and whether there is one."""
    flat = s["slots"].reshape(-1).long()
    where = torch.zeros(s["rows"] + 1, dtype=torch.int64, device=flat.device)
    where[torch.where(flat < 0, s["rows"], flat)] = torch.arange(1, flat.numel() + 1, device=flat.device)
    where = where[: s["rows"]]
    return (where - 1).clamp(min=0), where > 0


def _gate(z_of, act):
    """z and its derivative of act(g) = g * sigmoid(z(g))."""
    if act == "silu":
        return z_of, torch.ones_like(z_of)
    c = 2.0 * math.sqrt(2.0 / math.pi)
    return c * (z_of + 0.044715 * z_of * z_of * z_of), c * (1.0 + 3 * 0.044715 * z_of * z_of)


def _glu_values(gu, act):
    g, u = gu.double().chunk(2, dim=1)
    z, _ = _gate(g, act)
    return (g * u / (1.0 + torch.exp(-z))).float().to(torch.bfloat16)


def _plain_quantized(s, y, valid):
    """Quantized outputs of rows y of the padded layout (in 32 bits, rotated), zero where no row is."""
    case = s["case"]
    amax = s["amax"]
    if case["fmt"] == "nvfp4" and amax is None:
        amax = s["whole"].abs().amax()
    _, _, v, sg = _blocks(y, case["fmt"], case["strategy"], amax)
    v = torch.where(valid[:, None], v.reshape(y.shape), 0.0).to(torch.bfloat16)
    return {"values": v, "global_scale": sg.reshape(1) if sg is not None else None}


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "sort":
        counts, starts, slots = _plan(s["ids"], case["experts"])
        return {"counts": counts, "starts": starts, "slots": slots}
    choice, valid = _choice_of(s)
    token = choice // case["k"]
    if op == "quantize":
        y = _rotate(s["x"].float(), case["rot"])
        s = dict(s, whole=y)
        amax = s["amax"] if case["fmt"] != "nvfp4" or s["amax"] is not None else y.abs().amax()
        _, _, v, sg = _blocks(y, case["fmt"], case["strategy"], amax)
        v = torch.where(valid[:, None], v.reshape(y.shape).to(torch.bfloat16)[token], 0.0)
        return {"values": v, "global_scale": sg.reshape(1) if sg is not None else None}
    if op == "glu":
        h = torch.where(valid[:, None], _glu_values(s["gu"], case["act"]), 0.0)
        y = _rotate(h.float(), case["rot"])
        return _plain_quantized(dict(s, whole=y), y, valid)
    if op == "glu_bwd":
        dh = _rotate(s["dh"].float(), case["rot"])
        g, u = s["gu"].float().chunk(2, dim=1)
        z, dz = _gate(g, case["act"])
        p = 1.0 / (1.0 + torch.exp(-z))
        d = torch.cat((dh * u * (p + g * p * (1.0 - p) * dz), dh * g * p), 1)
        return torch.where(valid[:, None], d, 0.0).to(torch.bfloat16)
    if op == "gemm":
        fmt, cols = case["fmt"], case["cols"]
        a = _dequantized(s["a"], fmt, cols, torch.float32)[0]
        w = _dequantized(s["w"], fmt, cols, torch.float32)
        starts, counts = s["starts"].long(), s["counts"].long()
        lane = torch.arange(s["cap"], device=a.device)
        at = (starts[:-1, None] + lane).clamp(max=s["rows"] - 1)
        d = torch.matmul(a[at], w.transpose(1, 2))
        if fmt == "nvfp4":
            d = d * (s["a"][2] * s["w"][2])[:, None, None]
        out = torch.zeros(s["rows"] + 1, case["outs"], dtype=s["out"].dtype, device=a.device)
        out[torch.where(lane < counts[:, None], at, s["rows"])] = d.to(out.dtype)
        return out[: s["rows"]]
    flat = s["slots"].long()
    kept = (flat >= 0)[..., None]
    y = torch.where(kept, s["y"][flat.clamp(min=0)].float(), 0.0)
    w = s["weights"]
    if op == "combine":
        total = (y if w is None else y * w[..., None]).sum(1)
        return _rotate(total, case["rot"]).to(torch.float32 if case["f32"] else torch.bfloat16)
    g = s["g"].float()
    dy = torch.where(valid[:, None], w.reshape(-1)[choice][:, None] * g[token], 0.0).to(torch.bfloat16)
    return {"dy": dy, "dweights": (y * g[:, None]).sum(-1)}


def run(s):
    if not own:
        return _plain(s)
    import microscaling_fp4_quantization_bf16_b200 as fp4q
    case = s["case"]
    op = case["op"]
    if op == "sort":
        p = fp4q.expert_sort(s["ids"], case["experts"])
        return {"counts": p.counts, "starts": p.starts, "slots": p.slots}
    plan = fp4q.ExpertPlan(s["counts"], s["starts"], s["slots"], s["rows"])
    if op in ("quantize", "glu"):
        out = fp4q.Quantized(s["codes"], s["scales"], s["global_scale"], None, s["dq"])
        if op == "quantize":
            fp4q.expert_quantize(s["x"], plan, case["fmt"], case["strategy"], case["rot"], s["amax"], out=out)
        else:
            fp4q.glu_quantize(s["gu"], case["fmt"], case["strategy"], case["rot"], plan, case["act"], s["amax"], out=out)
        return {"values": out.dq, "global_scale": out.global_scale}
    if op == "glu_bwd":
        return fp4q.glu_bwd(s["gu"], s["dh"], plan, case["act"], case["rot"], out=s["out"])
    if op == "gemm":
        (ac, asc, ag), (wc, wsc, wg) = s["a"], s["w"]
        return fp4q.expert_gemm(ac[0], asc[0], ag, wc, wsc, wg, plan, case["fmt"], out=s["out"])
    if op == "combine":
        return fp4q.expert_combine(s["y"], plan, s["weights"], case["rot"], torch.float32 if case["f32"] else torch.bfloat16)
    dy, dw = fp4q.expert_combine_bwd(s["g"], s["y"], plan, s["weights"], out=s["out"])
    return {"dy": dy, "dweights": dw}


# ------------------------------------------------------------------------------------------------ what a pass needs

def work(case):
    op, t, k, e = case["op"], case["tokens"], case["k"], case["experts"]
    n = t * k
    live = n * (1.0 - DROP) if case["drop"] else n       # rows that hold a token
    if op == "sort":
        return {"bytes": n * (8 if case["wide"] else 4) + 4 * n + 8 * e, "flops": n}
    width = case.get("cols") or case.get("inner")
    per = 0.5 + 1.0 / _BLOCK[case["fmt"]] if "fmt" in case else 0.0
    if op == "quantize":
        twice = 2 if case["fmt"] == "nvfp4" and not case["calibrated"] else 1
        return {"bytes": 2 * t * width + live * width * (per + 2) + 4 * n, "flops": 10 * twice * t * width}
    if op == "glu":
        return {"bytes": live * width * (4 + per + 2) + 4 * n, "flops": 25 * live * width}
    if op == "glu_bwd":
        return {"bytes": live * width * 10 + 4 * n, "flops": 25 * live * width}
    if op == "gemm":
        weights = min(e, n) * case["outs"] * width * per
        return {"bytes": weights + live * (width * per + case["outs"] * (4 if case["f32"] else 2)), "flops": 2.0 * live * width * case["outs"]}
    if op == "combine":
        return {"bytes": 2 * live * width + t * width * (4 if case["f32"] else 2) + 8 * n, "flops": 2 * live * width}
    return {"bytes": 4 * live * width + 2 * t * width + 12 * n, "flops": 3 * live * width}


# ------------------------------------------------------------------------------------------------ in 64 bits

def _hadamard64(y, rot):
    if not rot:
        return y
    i = torch.arange(rot, device=y.device)
    bits = i[:, None] & i[None, :]
    odd = sum((bits >> b) & 1 for b in range(7)) % 2
    h = (1.0 - 2.0 * odd.double()) / math.sqrt(rot)
    return (y.reshape(-1, rot) @ h).reshape(y.shape)


def _nearest(a, mantissa, lowest, most):
    """a >= 0 to the nearest value of a small float format, ties to even: `mantissa` bits, smallest exponent `lowest`."""
    e = torch.floor(torch.log2(a.clamp(min=1e-300))).clamp(min=lowest)
    step = torch.exp2(e - mantissa)
    return (torch.round(a / step) * step).clamp(max=most)


def _exact_quantized(y, fmt, strategy, amax):
    b = _BLOCK[fmt]
    blocks = y.reshape(y.shape[0], -1, b)
    top = blocks.abs().amax(-1, keepdim=True)

    def values(scale):
        safe = torch.where(scale > 0, scale, 1.0)
        return torch.where(scale > 0, torch.sign(blocks) * _nearest((blocks / safe).abs(), 1, 0, 6.0) * scale, 0.0)

    if fmt == "mxfp4":
        scale = torch.exp2((torch.frexp(top).exponent - 3).double().clamp(-127, 127))
        return values(torch.where(top == 0, 2.0 ** -127, scale)).reshape(y.shape), None
    sg = amax.double() / 2688.0
    byte = [_nearest(top / (t * sg), 3, -6, 448.0) for t in (6.0, 4.0)]
    if strategy == "prevent_zero":
        byte[0] = byte[0].clamp(min=2.0 ** -9)
    v = values(byte[0] * sg)
    if strategy == "four_over_six":
        v4 = values(byte[1] * sg)
        v = torch.where((blocks - v4).square().sum(-1, keepdim=True) < (blocks - v).square().sum(-1, keepdim=True), v4, v)
    return v.reshape(y.shape), sg.reshape(1)


def exact(case, seed):
    op = case["op"]
    if op == "sort":
        return None
    s = prepare(case, seed)
    flat = s["slots"].reshape(-1).long()
    live = torch.nonzero(flat >= 0).reshape(-1)
    row, token = flat[live], live // case["k"]
    out64 = lambda width: torch.zeros(s["rows"], width, dtype=torch.float64, device="cuda")  # noqa: E731
    if op in ("quantize", "glu"):
        if op == "quantize":
            y = _hadamard64(s["x"].double(), case["rot"])
        else:
            g, u = s["gu"][row].double().chunk(2, dim=1)
            z, _ = _gate(g, case["act"])
            # the operator's own value in front of the quantizer is a bf16 number
            y = _hadamard64((g * u * torch.sigmoid(z)).float().to(torch.bfloat16).double(), case["rot"])
        amax = s["amax"] if s["amax"] is not None else y.abs().amax()
        v, sg = _exact_quantized(y, case["fmt"], case["strategy"], amax)
        out = out64(y.shape[1])
        out[row] = v[token] if op == "quantize" else v
        return {"values": out, "global_scale": sg}
    if op == "glu_bwd":
        g, u = s["gu"][row].double().chunk(2, dim=1)
        dh = _hadamard64(s["dh"][row].double(), case["rot"])
        z, dz = _gate(g, case["act"])
        p = torch.sigmoid(z)
        out = out64(2 * case["inner"])
        out[row] = torch.cat((dh * u * (p + g * p * torch.sigmoid(-z) * dz), dh * g * p), 1)
        return out
    if op == "gemm":
        out, starts, counts = out64(case["outs"]), s["starts"].tolist(), s["counts"].tolist()
        a = _dequantized(s["a"], case["fmt"], case["cols"], torch.float64)[0]
        for e, c in enumerate(counts):
            if c:
                one = tuple(None if x is None else x[e:e + 1] for x in s["w"])
                w = _dequantized(one, case["fmt"], case["cols"], torch.float64)[0]
                d = a[starts[e]:starts[e] + c] @ w.t()
                out[starts[e]:starts[e] + c] = d * s["a"][2].double() * s["w"][2][e].double() if case["fmt"] == "nvfp4" else d
        return out
    w = s["weights"]
    w = torch.ones(case["tokens"], case["k"], dtype=torch.float64, device="cuda") if w is None else w.double()
    part = w.reshape(-1)[live]
    if op == "combine":
        total = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
        return _hadamard64(total.index_add_(0, token, part[:, None] * s["y"][row].double()), case["rot"])
    g = s["g"].double()
    dy = out64(case["cols"])
    dy[row] = part[:, None] * g[token]
    dw = torch.zeros(case["tokens"] * case["k"], dtype=torch.float64, device="cuda")
    dw[live] = (g[token] * s["y"][row].double()).sum(1)
    return {"dy": dy, "dweights": dw.reshape(case["tokens"], case["k"])}

"""Plain definitions of the expert operators for the tests: numpy, 64 bits
(or, for codes and scales, the oracle)."""
import math

import numpy as np
import torch

import oracle

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def sort(ids, experts):
    """(counts, starts, slots) of int ids [T, k], by the definition."""
    flat = ids.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(experts)], np.int64)
    starts = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    slots = np.full(flat.size, -1, np.int64)
    for e in range(experts):
        at = np.nonzero(flat == e)[0]
        slots[at] = starts[e] + np.arange(at.size)
    return counts, starts, slots.reshape(ids.shape)


def bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


F = np.float32


def _rotate32(y, rot):
    """Butterflies of ascending distance in fp32, then one factor: the definition's rotation."""
    h = 1
    shape = y.shape
    while h < rot:
        p = y.reshape(-1, 2, h)
        y = np.stack([p[:, 0] + p[:, 1], p[:, 0] - p[:, 1]], 1)
        h *= 2
    return y.reshape(shape) * F(1 / math.sqrt(rot)) if rot else y.reshape(shape)


def _tree(v):
    while v.shape[-1] > 1:
        v = v[..., 0::2] + v[..., 1::2]
    return v[..., 0]


def _nvfp4(y, strategy, sg):
    """Codes, scale bytes and values of fp32 y [rows, cols] under s_g, one fp32 operation a step (the oracle's
    steps, which takes an abs-max only)."""
    v = y.reshape(y.shape[0], -1, 16)
    top = np.abs(v).max(-1, keepdims=True)
    e4m3 = np.array([oracle.e4m3_value(c) for c in range(0x7F)])
    mid = (e4m3[1:] + e4m3[:-1]) / 2

    def candidate(byte):
        S = e4m3.astype(F)[byte] * sg
        with np.errstate(divide="ignore"):
            r = np.where(S == 0, F(0), np.minimum(F(1) / S, np.finfo(F).max))
        a = np.abs(v * r).astype(np.float64)
        steps = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0])
        m = sum((a >= t) if i % 2 else (a > t) for i, t in enumerate(steps))
        code = np.where(S == 0, 0, m + 8 * np.signbit(v))
        w = E2M1.astype(F)[code] * S
        d = v - w
        return byte, code, w, _tree(d * d)[..., None]

    def nearest(target):
        x = (top / (sg * F(target))).astype(np.float64)
        k = np.searchsorted(mid, x, side="left")            # ties: below, then up to the even code
        tie = (k < 126) & (np.append(mid, np.inf)[np.minimum(k, 126)] == x) & (k % 2 == 1)
        return np.minimum(k + tie, 0x7E)
    best = candidate(nearest(6))
    if strategy == "prevent_zero":
        best = candidate(np.maximum(best[0], 1))
    elif strategy == "four_over_six":
        other = candidate(nearest(4))
        take = other[3] < best[3]
        best = [np.where(take, o, b) for o, b in zip(other, best)]
    elif strategy == "brute_force":
        best = candidate(np.full_like(best[0], 1))
        for c in range(2, 0x7F):
            other = candidate(np.full_like(best[0], c))
            take = other[3] < best[3]
            best = [np.where(take, o, b) for o, b in zip(other, best)]
    byte, code, w, _ = best
    code = code.reshape(y.shape).astype(np.uint8)
    return {"codes": code[:, 0::2] | (code[:, 1::2] << 4), "scales": byte[..., 0].astype(np.uint8),
            "global_scale": sg, "dq": w.reshape(y.shape).astype(F)}


def quantize(x_bits, fmt, strategy, rot, amax=None):
    """Codes, row-major scales, values (fp32) and s_g of bf16 bit patterns: the oracle's for a given abs-max and for
    MXFP4; for NVFP4 without one the same steps under s_g = abs-max * fp32(1 / 2688)."""
    if fmt == "mxfp4" or amax is not None:
        return oracle.quantize(x_bits, fmt, BLOCK[fmt], strategy, rot, dq="f32", global_amax=amax)
    y = _rotate32((x_bits.astype(np.uint32) << 16).view(F), rot)
    return _nvfp4(y, strategy, np.abs(y).max() * F(1 / 2688))


def mma_rows(flat, rows, blocks):
    """MMA-layout scale bytes -> [rows, padded blocks]."""
    pad = -(-blocks // 4) * 4
    a = np.asarray(flat).reshape(-1, pad // 4, 32, 4, 4).transpose(0, 3, 2, 1, 4)
    return a.reshape(-1, pad)[:rows]


def values(codes, flat_scales, rows, cols, fmt):
    """float64 values of packed codes under MMA-layout scales, without s_g."""
    b = BLOCK[fmt]
    c = np.stack([codes & 15, codes >> 4], -1).reshape(rows, cols // b, b)
    s = mma_rows(flat_scales, rows, cols // b)[:, :cols // b].astype(np.int64)
    if fmt == "mxfp4":
        scale = np.exp2((s - 127).astype(np.float64))
    else:
        e, m = s >> 3, s & 7
        scale = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * np.exp2((e - 7).astype(np.float64)))
    return (E2M1[c] * scale[..., None]).reshape(rows, cols)


def gate(g, act):
    """z(g) and z'(g) of act(g) = g sigmoid(z(g))."""
    if act == "silu":
        return g, np.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g ** 2)


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-z))


def glu(gu_bits, act):
    """bf16 bits of h = bf16(fp32(a(g) u)) from bf16 bits [rows, 2 cols]."""
    gu = (gu_bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    g, u = np.split(gu, 2, axis=1)
    h = (g * u * sigmoid(gate(g, act)[0])).astype(np.float32)
    return bits(torch.from_numpy(h).to(torch.bfloat16))


def hadamard(rot):
    h = np.ones((1, 1))
    while h.shape[0] < rot:
        h = np.block([[h, h], [h, -h]])
    return h / math.sqrt(rot)


def rotate(y, rot):
    if not rot:
        return y
    return (y.reshape(-1, rot) @ hadamard(rot)).reshape(y.shape)


def to64(t):
    return t.float().cpu().numpy().astype(np.float64)


def route(tokens, k, experts, seed, drop=0.0, used=None):
    """Choices [tokens, k] (int64): random experts among the first `used`, some dropped."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts if used is None else used, (tokens, k))
    ids[rng.random((tokens, k)) < drop] = -1
    return ids

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


def quantize(x_bits, fmt, strategy, rot, amax=None):
    """Oracle codes, row-major scales, values (fp32) and s_g of bf16 bit patterns."""
    return oracle.quantize(x_bits, fmt, BLOCK[fmt], strategy, rot, dq="f32",
                           **({} if amax is None else {"global_amax": amax}))


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

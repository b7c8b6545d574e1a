"""Plain 64-bit references (numpy, CPU) of the optimiser and quantised-linear operators."""
from __future__ import annotations

import numpy as np

BLOCK = 32
M32 = np.uint64(0xFFFFFFFF)


# ---- 4-bit weights -----------------------------------------------------------------------------

def int4_place(cols):
    """Word of a row and low bit of each column's nibble."""
    c = np.arange(cols)
    word = c // 128 * 16 + 4 * (c % 32 // 8) + c % 128 // 32
    return word, 4 * (c % 8 // 2 + 4 * (c % 2))


def int4_pack(codes):
    rows, cols = codes.shape
    word, shift = int4_place(cols)
    q = np.zeros((rows, (cols + 127) // 128 * 16), np.uint32)
    for c in range(cols):
        q[:, word[c]] |= codes[:, c].astype(np.uint32) << np.uint32(shift[c])
    return q


def int4_unpack(q, cols):
    word, shift = int4_place(cols)
    return (q[:, word] >> shift.astype(np.uint32)) & np.uint32(15)


def int4_quantize(w, group, with_zeros):
    """(codes [rows, cols], scales fp32, zeros or None) by exact division and rounding."""
    w = np.asarray(w, np.float64)
    rows, cols = w.shape
    groups = -(-cols // group)
    codes = np.zeros((rows, cols), np.uint32)
    scales, zeros = np.zeros((rows, groups), np.float32), np.zeros((rows, groups), np.uint8)
    for r in range(rows):
        for g in range(groups):
            x = w[r, g * group:(g + 1) * group]
            if not np.all(np.isfinite(x)):
                scales[r, g] = np.nan
                zeros[r, g] = 0
                codes[r, g * group:(g + 1) * group] = 0 if with_zeros else 8
                continue
            lo, hi = min(x.min(), 0.0), max(x.max(), 0.0)
            s = np.float32((hi - lo) / 15) if with_zeros else np.float32(max(hi, -lo) / 7)
            scales[r, g] = s
            s = np.float64(s)
            z = (min(np.rint(-lo / s), 15.0) if s > 0 else 0.0) if with_zeros else 8.0
            zeros[r, g] = z
            q = np.rint(x / s) if s > 0 else np.zeros_like(x)
            codes[r, g * group:(g + 1) * group] = np.clip(q + z, 0, 15)
    return codes, scales, zeros if with_zeros else None


def int4_weights(codes, scales, zeros, group):
    g = np.arange(codes.shape[1]) // group
    z = 8.0 if zeros is None else zeros.astype(np.float64)[:, g]
    return (codes.astype(np.float64) - z) * scales.astype(np.float64)[:, g]


# ---- trellis-coded weights -----------------------------------------------------------------------

def code_states(code, n, k, L):
    """States [chains, L]: the n-bit windows of each chain's bit string at bits k t."""
    bits = np.unpackbits(code.astype(">u4").view(np.uint8), axis=1)
    s = np.zeros((code.shape[0], L), np.int64)
    at = k * np.arange(L)
    for i in range(n):
        s = 2 * s + bits[:, at + i]
    return s


# ---- AdamW ---------------------------------------------------------------------------------------

def mix(x):
    x = np.asarray(x, np.uint64) & M32
    x ^= x >> np.uint64(16)
    x = (x * np.uint64(0x6A09E667)) & M32
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(0xBB67AE85)) & M32
    return x ^ (x >> np.uint64(16))


def dithers(first, count, step, seed):
    key = mix((mix(np.uint64(seed & 0xFFFFFFFF)) + np.uint64(step)) & M32)
    at = np.arange(first, first + count, dtype=np.uint64)
    h = mix(((at & M32) * np.uint64(0x9E3779B1) + (at >> np.uint64(32)) * np.uint64(0x85EBCA6B) + key) & M32)
    return ((h & np.uint64(0xFFFF)).astype(np.float64) + 0.5) / 65536, ((h >> np.uint64(16)).astype(np.float64) + 0.5) / 65536


def e4m3_values():
    """The 256 values of e4m3 codes."""
    c = np.arange(256)
    e, n = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8.0 + n) * 2.0 ** (e - 10), n * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def encode(x, d, least):
    """(values, exponents b) of blocks x [blocks, 32] with dithers d."""
    fine = np.isfinite(x)
    a = np.where(fine, np.abs(x), 0.0)
    top = a.max(axis=1, keepdims=True)
    b = np.where(top > 0, np.clip(np.frexp(top)[1] - 1 - 7 + 127, 0, 254), 0)
    y = np.ldexp(a, 127 - b)
    e = np.maximum(np.frexp(y)[1] - 1, -6)
    n = np.floor(np.ldexp(y, 3 - e) + d)
    n = np.where(y > 0, np.maximum(n, least), 0.0)
    return np.where(fine, np.sign(x) * np.ldexp(n, e - 3), np.nan), b[:, 0].astype(np.uint8)


def adamw(p, g, m, second, h, bits, first=0, scales=None):
    """One tensor's step. bits = 32: (p', m', v'); bits = 8: m, second are code values and scales their
    exponents; (p', m values, r values, m exponents, r exponents)."""
    p, g = np.asarray(p, np.float64), np.asarray(g, np.float64)
    n = p.size
    b1, b2, t = h["beta1"], h["beta2"], h["step"]
    m, second = np.asarray(m, np.float64)[:n], np.asarray(second, np.float64)[:n]
    if bits == 8:
        block = np.arange(n) // BLOCK
        m = np.ldexp(m, scales[0].astype(int)[block] - 127)
        second = np.ldexp(second, scales[1].astype(int)[block] - 127) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * second + (1 - b2) * (g * g)
    with np.errstate(all="ignore"):
        by = (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + h["eps"])
    new = p - h["lr"] * h["weight_decay"] * p - h["lr"] * by
    if bits == 32:
        return new, m, v
    pad = -n % BLOCK
    blocks = lambda a: np.pad(a, (0, pad)).reshape(-1, BLOCK)  # noqa: E731
    dm, dr = dithers(first, n + pad, t, h["seed"])
    with np.errstate(all="ignore"):
        mv, mb = encode(blocks(m), dm.reshape(-1, BLOCK), 0)
        rv, rb = encode(blocks(np.sqrt(v)), dr.reshape(-1, BLOCK), 1)
    return new, mv.reshape(-1)[:n], rv.reshape(-1)[:n], mb, rb

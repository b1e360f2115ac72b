"""Definitions of the attention-side operators in numpy: rotary positions, the
block quantizers and byte layout of the paged key/value cache, and attention of
one token over it.  Arithmetic is binary64 except the quantizers' quotients,
which are defined in binary32.  Independent of the library's code.
"""
from __future__ import annotations

import numpy as np

KINDS = {"F16": 1, "Q8_0": 8, "Q4_0": 2}
BLOCK_BYTES = {"F16": 64, "Q8_0": 34, "Q4_0": 18}  # one row of 32 elements
UNIT = {"F16": 2048, "Q8_0": 1024, "Q4_0": 512}    # codes of 32 elements x 32 tokens


def page_bytes(kind, page_size, n_kv, head_dim):
    return page_size * n_kv * head_dim // 32 * BLOCK_BYTES[kind]


# -- rotary positions --------------------------------------------------------
def rope(x, pos, freqs, layout="half", mscale=1.0):
    """x [T, H, D] rotated, in binary64."""
    y = x.astype(np.float64).copy()
    n = 2 * len(freqs)
    phi = (pos.astype(np.float64)[:, None] * freqs[None, :])[:, None, :]
    a = np.arange(n // 2) if layout == "half" else 2 * np.arange(n // 2)
    b = a + (n // 2 if layout == "half" else 1)
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a] = mscale * (u * np.cos(phi) - v * np.sin(phi))
    y[..., b] = mscale * (u * np.sin(phi) + v * np.cos(phi))
    return y


def rope_bound(x, n_rot, layout="half", mscale=1.0):
    """mscale (|x_a| + |x_b|) of each element's pair; 0 for passing elements."""
    x = np.abs(x.astype(np.float64))
    y = np.zeros_like(x)
    half = n_rot // 2
    if layout == "half":
        s = x[..., :half] + x[..., half:n_rot]
        y[..., :half], y[..., half:n_rot] = s, s
    else:
        s = x[..., 0:n_rot:2] + x[..., 1:n_rot:2]
        y[..., 0:n_rot:2], y[..., 1:n_rot:2] = s, s
    return abs(mscale) * y


# -- quantizers --------------------------------------------------------------
def f16_up(d):
    """The smallest float16 >= d (d >= 0, float32), at most 65504."""
    h = np.minimum(d, np.float32(65504)).astype(np.float16)
    low = (h.astype(np.float32) < d) & (h < np.float16(65504))
    return np.where(low, (h.view(np.uint16) + 1).astype(np.uint16).view(np.float16), h)


def quantize(kind, x):
    """Stored codes (uint8, or the halves of F16) and float16 scales of x [..., D] float32."""
    x = x.astype(np.float32)
    if kind == "F16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16), None
    blk = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        hi, lo = blk.max(-1), blk.min(-1)
        bad = ~np.isfinite(blk).all(-1)
        d = np.abs(np.maximum(hi, -lo)) / np.float32(127 if kind == "Q8_0" else 8)
        h = f16_up(np.where(bad, np.float32(0), d).astype(np.float32))
        if kind == "Q4_0":
            h = np.where((hi >= -lo) & (h != 0), -h, h)
        h32 = h.astype(np.float32)[..., None]
        q = np.where((h32 == 0) | bad[..., None], np.float32(0), blk / np.where(h32 == 0, np.float32(1), h32))
        q = np.rint(q)
    q = np.clip(q, -127, 127) + 128 if kind == "Q8_0" else np.clip(q + 8, 0, 15)
    h = np.where(bad, np.float16(np.nan), h)
    return q.astype(np.uint8).reshape(x.shape), h


def dequantize(kind, codes, h):
    """Exact values in binary64."""
    if kind == "F16":
        return codes.astype(np.float64)
    blk = codes.astype(np.float64).reshape(*codes.shape[:-1], -1, 32) - (128 if kind == "Q8_0" else 8)
    return (blk * h.astype(np.float64)[..., None]).reshape(codes.shape)


# -- byte layout -------------------------------------------------------------
def code_at(kind, is_v, r, d):
    """Byte offset in a group of element d of token r (Q4_0: and the nibble)."""
    b, c = d // 32, d % 32
    base = b * UNIT[kind]
    i, m = 4 * (r // 8) + r % 4, (r // 4) % 2
    if not is_v:
        if kind == "F16":
            return base + ((4 * m + c // 8) * 16 + i) * 16 + 2 * (c % 8)
        if kind == "Q8_0":
            return base + ((16 * (c // 8) + i) * 2 + m) * 8 + c % 8
        return base + ((16 * (c % 16 // 4) + i) * 2 + m) * 4 + c % 4
    if kind == "F16":
        return base + ((4 * (c // 16) + r // 8) * 16 + c % 16) * 16 + 2 * (r % 8)
    if kind == "Q8_0":
        return base + ((16 * (r // 8) + c % 16) * 2 + c // 16) * 8 + r % 8
    return base + (16 * (r // 8) + c % 16) * 8 + r % 8


def store(kind, is_v, pages, page_size, slot, codes, h):
    """Writes one token's codes [n_kv, D] and scales [n_kv, D / 32] into pages [n_pages, page_bytes] uint8."""
    n_kv, D = codes.shape
    page, off = divmod(slot, page_size)
    g, r = divmod(off, 32)
    gb = 32 * (D // 32) * BLOCK_BYTES[kind]
    d = np.arange(D)
    at = code_at(kind, is_v, r, d)
    for head in range(n_kv):
        p = pages[page, (head * (page_size // 32) + g) * gb:][:gb]
        if kind == "F16":
            raw = codes[head].view(np.uint16)
            p[at], p[at + 1] = raw & 255, raw >> 8
            continue
        if kind == "Q8_0":
            p[at] = codes[head]
        else:
            for x in (0, 1):
                sel = d[(d % 32) // 16 == x]
                keep = p[at[sel]] & (0xF0 if x == 0 else 0x0F)
                p[at[sel]] = keep | (codes[head][sel] << (4 * x))
        sat = (D // 32) * UNIT[kind] + (np.arange(D // 32) * 32 + r) * 2
        raw = h[head].view(np.uint16)
        p[sat], p[sat + 1] = raw & 255, raw >> 8


def load(kind, is_v, pages, page_size, slot, n_kv, D):
    """Exact values [n_kv, D] of one token."""
    page, off = divmod(slot, page_size)
    g, r = divmod(off, 32)
    gb = 32 * (D // 32) * BLOCK_BYTES[kind]
    d = np.arange(D)
    at = code_at(kind, is_v, r, d)
    out = np.empty((n_kv, D))
    for head in range(n_kv):
        p = pages[page, (head * (page_size // 32) + g) * gb:][:gb].astype(np.uint16)
        if kind == "F16":
            out[head] = (p[at] | p[at + 1] << 8).astype(np.uint16).view(np.float16)
            continue
        c = p[at] if kind == "Q8_0" else p[at] >> (4 * (d % 32 // 16)) & 15
        sat = (D // 32) * UNIT[kind] + (np.arange(D // 32) * 32 + r) * 2
        h = (p[sat] | p[sat + 1] << 8).astype(np.uint16).view(np.float16)
        out[head] = dequantize(kind, c[None].astype(np.uint8), h[None])[0]
    return out


# -- attention ---------------------------------------------------------------
def attend(q, k, v, scale, sink=None, f16=True, counts=None):
    """One query head q [D] over k, v [n, D] (binary64), token t counts[t] times
    (None: once): the output and its tolerance, without the output's rounding: the
    header's bound without its terms for far smaller elements (f16_floor, and a
    query's 2^-13 max |q|), f16 queries held to the f32 ones' constant for scores,
    2^-20 instead of the documented 2^-17."""
    n, D = k.shape
    if n == 0:
        return np.zeros(D), np.zeros(D)
    q = q.astype(np.float64)
    s = scale * (k @ q)
    top = s.max() if sink is None else max(s.max(), float(sink))
    p = np.exp(s - top) * (1 if counts is None else counts)
    w = p / (p.sum() + (0 if sink is None else np.exp(float(sink) - top)))
    aq = np.abs(q).reshape(-1, 32).sum(-1)
    ak = np.abs(k).reshape(n, -1, 32).max(-1)
    e = 2.0 ** -20 * (abs(scale) * (ak @ aq).max() + np.abs(s).max() + 40)
    r = 2.0 ** -18 + (2.0 ** -11 if f16 else 0)
    return w @ v, (r + 2 * e) * (w @ np.abs(v))


def f16_floor(v, scales, w):
    """What f16 weights may lose in each element beyond attend's tolerance: v [n, D] exact values, scales [n, D / 32]
    of their blocks (None: F16), w [n] exact weights, token 0 of the arrays at a multiple of eight."""
    n, D = v.shape
    pad = -n % 8
    top = np.pad(w, (0, pad)).reshape(-1, 8).max(-1)
    d = np.ones((n, 1)) if scales is None else np.abs(scales.astype(np.float64))
    big = np.pad(d.max(-1), (0, pad)).reshape(-1, 8).max(-1)
    d = np.where(d == 0, 1, d).repeat(D // d.shape[1], -1)
    return 2.0 ** -39 * (top * big).max() * np.abs(v / d).sum(0)

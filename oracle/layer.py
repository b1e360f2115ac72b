"""What stands around a layer's products, in numpy and binary64: the norm with
the residual's addition, the choice of experts, and a product's epilogue.

TEST INFRASTRUCTURE ONLY.  Only ``tests/`` and ``__graft_entry__.smoke()`` may
use it.  It shares no code with the HIP library and never calls it.  Model
semantics beyond the pages, like the expert FFN; the definitions are those
of include/qmm.h.
"""
from __future__ import annotations

import math

import numpy as np

from . import int8

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
# Where an activation has its only minimum (between two rising parts), to 1e-9.
LOWEST = {"silu": -1.278464543, "gelu": -0.751791524, "gelu_tanh": -0.752461422}
# Bounds of |act'|: of silu 1.0998 (near 2.4), of both gelus 1.129 (near 1.41).
SLOPE = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13}

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def rmsnorm(x, residual=None, weight=None, eps=1e-6):
    """(h, y): the sum in float32 and the normed rows in float64, over the last axis."""
    h = np.asarray(x).astype(np.float32)
    if residual is not None:
        with np.errstate(over="ignore"):
            h = h + np.asarray(residual).astype(np.float32)
    v = h.astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        size = np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + float(np.float32(eps)))
        y = np.where(size == 0, 0.0, v / size)
        if weight is not None:
            y = y * np.asarray(weight).astype(np.float64)
    return h, y


def lane_order(kind) -> np.ndarray:
    """Position of element e of a block among its 32 codes: element order for Q8_0 weights; for the others position 8 G
    + 4 h + j holds element 16 h + 4 G + j."""
    e = np.arange(32)
    return e if kind == "Q8_0" else 8 * (e % 16 // 4) + 4 * (e // 16) + e % 4


def eight_bits(kind, y):
    """(codes in the lane order of `kind`, scales, code sums) of f32 rows y [T][D]."""
    q, d = int8.quantize(np.asarray(y, dtype=np.float32))
    T, D = q.shape
    blocks = q.reshape(T, D // 32, 32)
    codes = np.empty_like(blocks)
    codes[:, :, lane_order(kind)] = blocks
    return codes.reshape(T, D), d, blocks.astype(np.int32).sum(-1)


def activation(act, v):
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(over="ignore"):
        if act in ("none", None):
            return v
        if act == "relu":
            return np.maximum(v, 0.0)
        if act == "silu":
            return v / (1.0 + np.exp(-v))
        if act == "gelu":
            return 0.5 * v * _erfc(-v / math.sqrt(2.0))
        if act == "gelu_tanh":
            return v / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    raise KeyError(act)


def moved(act, u, err):
    """How far act(v) can be from act(u) for v within err of u.  Between its minimum and either side an activation only
    falls or rises, so the farthest are the ends or the minimum."""
    y = activation(act, u)
    far = np.maximum(np.abs(activation(act, u - err) - y), np.abs(activation(act, u + err) - y))
    if act in LOWEST:
        low = LOWEST[act]
        far = np.where(np.abs(u - low) <= err + 1e-9, np.maximum(far, np.abs(activation(act, low) - y)), far)
    return far


def epilogue(v, err, bias=None, act="none", mul=None, residual=None, f16=False):
    """(out, tol) for sums v that are known to `err`: the epilogue in binary64, and what the sums' error and f32 steps
    (2^-24 relative each, for the activation 2^-20 or 2^-126 absolute) make of it, beside the result's own rounding."""
    b = 0.0 if bias is None else np.asarray(bias, dtype=np.float64)
    u = v + b
    err = err + 2.0 ** -24 * np.abs(u)
    y = activation(act, u)
    tol = moved(act, u, err)
    if act not in ("none", None, "relu"):
        tol = tol + 2.0 ** -20 * (np.abs(y) + tol) + 2.0 ** -126
    if mul is not None:
        m = np.asarray(mul).astype(np.float64)
        y, tol = y * m, tol * np.abs(m)
        tol = tol + 2.0 ** -24 * np.abs(y)
    if residual is not None:
        y = y + np.asarray(residual).astype(np.float64)
        tol = tol + 2.0 ** -24 * np.abs(y)
    tol = tol * (1 + 2.0 ** -20) + 2.0 ** -140
    if f16:
        tol = tol * (1 + 2.0 ** -11) + 2.0 ** -11 * np.abs(y) + 2.0 ** -25
    return y, tol


def route(logits, topk, score="softmax", bias=None, n_group=1, topk_group=1, group_top=1, normalize=True, scale=1.0,
          slots=None):
    """(ids int32, weights float64) [M][topk], one row and one expert at a time."""
    logits = np.asarray(logits)
    M, E = logits.shape
    ids = np.full((M, topk), -1, np.int32)
    weights = np.zeros((M, topk))
    size = E // n_group
    for t in range(M):
        if slots is not None and slots[t] < 0:
            continue
        l = [float(v) for v in logits[t]]
        there = [e for e in range(E) if l[e] > -math.inf]  # neither NaN nor -inf
        if score == "softmax":
            top = max((l[e] for e in there), default=0.0)
            # (Infinite logits share all of it.)
            ex = {e: 1.0 if l[e] == top else math.exp(l[e] - top) for e in there}
            total = math.fsum(ex.values())
            s = {e: ex[e] / total for e in there}
        else:
            s = {e: 1.0 / (1.0 + math.exp(-l[e])) if l[e] >= -700 else math.exp(max(l[e], -1e4)) for e in there}
        sums = n_group > 1 and group_top == 2
        if bias is None and not sums:
            c = {e: l[e] for e in there}  # in the scores' order, ties and all
        else:
            c = {e: s[e] + (0.0 if bias is None else float(bias[e])) for e in there}
        c = {e: v for e, v in c.items() if v > -math.inf}
        if n_group > 1:
            value = {}
            for g in range(n_group):
                mine = sorted((c[e] for e in range(g * size, (g + 1) * size) if e in c), reverse=True)
                if mine:
                    value[g] = sum(mine[:group_top])
            kept = sorted(value, key=lambda g: (-value[g], g))[:topk_group]
            c = {e: v for e, v in c.items() if e // size in kept}
        chosen = sorted(c, key=lambda e: (-c[e], e))[:topk]
        if not chosen:
            continue
        if normalize:
            # Ratios of scores relative to the largest: nothing vanishes with them.
            lead = max(l[e] for e in chosen)
            if score == "softmax":
                w = [1.0 if l[e] == lead else math.exp(l[e] - lead) for e in chosen]
            elif lead < 0:
                w = [math.exp(l[e] - lead) / (1.0 + math.exp(l[e])) for e in chosen]
            else:
                w = [s[e] for e in chosen]
            w = [v / math.fsum(w) for v in w]
        else:
            w = [s[e] for e in chosen]
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = np.array(w) * float(np.float32(scale))
    return ids, weights

"""Test infrastructure: the 4-bit layers in plain numpy, FP64, from their
definitions (include/tern.h): packing, product, routing, routed experts, and
the error bounds the GPU results are held to.  Shares no code with the HIP
path."""
from __future__ import annotations

import numpy as np

# A product q * x of an integer below 2^8 and an FP16 value is exact in FP32.
# An FP32 addition is off by one unit at most (2^-23; half of it if rounded to
# nearest, which the matrix instructions need not do inside).
ADD = 2.0 ** -23


def pack(q):
    """uint8 codes [..., k] -> bytes [..., k/2]: offset o of eight in bits
    16 (o % 2) + 4 (o // 2) of a little-endian word."""
    q = np.asarray(q, np.uint32)
    word = np.zeros((*q.shape[:-1], q.shape[-1] // 8), np.uint32)
    for o in range(8):
        word |= q[..., o::8] << np.uint32(16 * (o % 2) + 4 * (o // 2))
    return word.astype("<u4").view(np.uint8)


def dequant(q, scale, zero, group):
    z = 8.0 if zero is None else np.repeat(zero.astype(np.float64), group, axis=-1)
    return (q.astype(np.float64) - z) * np.repeat(scale.astype(np.float64), group, axis=-1)


def half_step(y, out):
    """Half a step of the output type at y."""
    return np.abs(y) * 2.0 ** -11 + 2.0 ** -25 if out == "f16" else np.abs(y) * 2.0 ** -24 + 2.0 ** -150


def adds(k, group):
    """Additions a product passes through: at most G inside its group, one for
    each group, 64 joining wavefronts and K parts; scaling rounds once more."""
    return group + k // group + 65


def gemm(q, scale, zero, group, x):
    """(y, B, bound of the FP32 sums' error): B = sum |w x|."""
    w = dequant(q, scale, zero, group)
    x = x.astype(np.float64)
    y, b = x @ w.T, np.abs(x) @ np.abs(w).T
    return y, b, adds(q.shape[1], group) * ADD * b


def route(logits, topk, score="softmax", bias=None, groups=1, best=1, keep=1, renorm=True, scale=1.0):
    """One token at a time, by sorting.  (ids int32, weights fp64.)"""
    m, experts = logits.shape
    ids = np.full((m, topk), -1, np.int32)
    weights = np.zeros((m, topk))
    size = experts // groups
    for t in range(m):
        l = [min(float(v), float(np.finfo(np.float32).max)) if v == v else -np.inf for v in logits[t].astype(np.float64)]
        live = [e for e in range(experts) if l[e] > -np.inf]
        if not live:
            continue
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s = {e: 1.0 / (1.0 + np.exp(-l[e])) for e in live}
        else:
            top = max(l)
            total = sum(np.exp(l[e] - top) for e in live)
            s = {e: np.exp(l[e] - top) / total for e in live}
        # without a bias the order is the logits'; two experts' scores are summed as such
        key = l if bias is None else {e: s[e] + float(bias[e]) for e in live}
        key = {e: key[e] for e in live if key[e] == key[e] and key[e] > -np.inf}
        if groups > 1:
            judged = s if bias is None and best == 2 else key
            sums = []
            for g in range(groups):
                mine = sorted((judged[e] for e in key if e // size == g), reverse=True)[:best]
                sums.append(sum(mine) if mine else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-sums[g], g))[:keep]
            key = {e: v for e, v in key.items() if e // size in kept}
        chosen = sorted(key, key=lambda e: (-key[e], e))[:topk]
        g = np.array([s[e] for e in chosen])
        if renorm and g.sum() > 0:
            g = g / g.sum()
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = g * scale
    return ids, weights


def experts(up, down, group, x, ids, gates, parts=1):
    """up, down: (q, scale, zero) stacks.  (y, bound without the output's own
    rounding.)  The inner values' error: the FP32 sums of gate and up (silu's
    slope is below 1.1), the exponential ((|g| + 4) 2^-22 relative), and their
    rounding to a BF16 value and `parts` more (1, or 2 for up to 32 slots),
    each of what the ones before leave: the first is off by 2^-8, and a rest
    lies a binade lower than what it may be off by, so each one more brings
    nine bits.  A product of a value and a code that FP32 cannot hold is lost
    (2^-69 of a code's step).  This reaches y through |Wd|; the down product's
    sums (every value's parts are added) and the slots' add theirs."""
    m, topk = ids.shape
    count = up[0].shape[0]
    y = np.zeros((m, down[0].shape[1]))
    err = np.zeros_like(y)
    for t in range(m):
        for j in range(topk):
            e = ids[t, j]
            if not 0 <= e < count:
                continue
            of = lambda w: (w[0][e], w[1][e], None if w[2] is None else w[2][e])
            gu, _, d = gemm(*of(up), group, x[t:t + 1])
            i = gu.shape[1] // 2
            g, u, dg, du = gu[0, :i], gu[0, i:], d[0, :i], d[0, i:]
            with np.errstate(over="ignore"):
                silu = g / (1 + np.exp(-g))
            h = silu * u
            dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + np.abs(h) * (np.abs(g) + 4) * 2.0 ** -22
            dh = dh + (np.abs(h) + dh) * 2.0 ** (-8 - 9 * parts) + 2.0 ** -69
            w = dequant(*of(down), group)
            gate = float(gates[t, j])
            y[t] += gate * (w @ h)
            b = np.abs(w) @ (np.abs(h) + dh) * (1 + 2.0 ** -7)
            err[t] += abs(gate) * (np.abs(w) @ dh + (adds(w.shape[1], group) + parts * group + topk + 1 + parts) * ADD * b)
    return y, err

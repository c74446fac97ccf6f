"""Plain fp64 oracle of rotary positions, the 8-bit cache and attention over
it.  Test infrastructure only; shares no code with the HIP path.

A cache is codes int64 [pages][heads][64][dim] and scales fp64 [pages][heads]
in the order of tokens and dimensions; pack and unpack give the byte order of
tern_kv.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


# ---------------------------------------------------------------- bytes
def place(dim: int, keys: bool) -> np.ndarray:
    """Byte offset of every (token, dimension) in a page's 64 * dim bytes."""
    at = np.empty((PAGE, dim), np.int64)
    for token in range(PAGE):
        for d in range(dim):
            if keys:
                a, t, i = token // 16, token // 4 % 4, token % 4
                c, r, b = d // 64, d // 16 % 4, d % 16
                at[token, d] = ((4 * c + t) * 64 + 16 * r + 4 * a + i) * 16 + b
            else:
                a, j = divmod(token, 16)
                c, e = divmod(d, 16)
                at[token, d] = ((4 * c + a) * 16 + e) * 16 + j
    return at


def pack(codes, keys: bool) -> np.ndarray:
    """Codes [pages][heads][64][dim] to bytes [pages][heads][64 * dim]."""
    p, h, _, dim = codes.shape
    out = np.empty((p, h, PAGE * dim), np.uint8)
    out[:, :, place(dim, keys)] = codes + 128
    return out


def unpack(raw, dim: int, keys: bool) -> np.ndarray:
    """The inverse, int64."""
    return np.asarray(raw).reshape(*np.shape(raw)[:2], -1)[:, :, place(dim, keys)].astype(np.int64) - 128


# ---------------------------------------------------------------- positions
def rope(x, pos, freq, interleaved=False, amp=1.0, norm=None, eps=1e-6) -> np.ndarray:
    """x [m][heads][dim] turned, fp64."""
    y = np.asarray(x, np.float64).copy()
    if norm is not None:
        y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * np.asarray(norm, np.float64)
    out = y.copy()
    half = len(freq)
    for i in range(half):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = np.asarray(pos, np.float64) * freq[i]
        c, s = amp * np.cos(angle)[:, None], amp * np.sin(angle)[:, None]
        out[..., lo] = y[..., lo] * c - y[..., hi] * s
        out[..., hi] = y[..., hi] * c + y[..., lo] * s
    return out


def frequencies(rot, base, scaling="plain", factor=1.0, low=1.0, high=32.0, trained=4096):
    """(frequencies, amplitude): straight from the definitions."""
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" and rot > 2 else base
        f = b ** (-2 * i / rot)
        if scaling == "linear":
            f = f / factor
        if scaling in ("ramp", "waves"):
            if scaling == "waves":
                share = (trained * f / (2 * np.pi) - low) / (high - low)
            else:
                edge = [rot * np.log(trained / (t * 2 * np.pi)) / (2 * np.log(base)) for t in (high, low)]
                first, last = max(0, np.floor(edge[0])), min(rot - 1, np.ceil(edge[1]))
                share = 1 - (i - first) / max(last - first, 1e-3)
            share = min(1.0, max(0.0, share))
            f = share * f + (1 - share) * f / factor
        out.append(f)
    return np.array(out), 0.1 * np.log(factor) + 1 if scaling == "ramp" else 1.0


# ---------------------------------------------------------------- the cache
def least_scale(most: float) -> float:
    """The smallest number of 8 significant bits with most <= 127 of it."""
    if most == 0:
        return 0.0
    exponent = np.floor(np.log2(most / 127)) - 7
    step = 2.0 ** exponent
    return float(np.ceil(most / 127 / step) * step)


def spans(start, length, count, rows, max_rows):
    """(first row, rows taken, position of the first) of every sequence."""
    out = []
    for s in range(count):
        first = s * max_rows if start is None else start[s]
        n = max_rows if start is None else start[s + 1] - start[s]
        out.append((first, min(n, max_rows), length[s] - n))
    return out


def page_of(table, pages, s, position):
    p = position // PAGE
    if position < 0 or p >= len(table[s]) or not 0 <= table[s][p] < pages:
        return None
    return int(table[s][p])


def write(codes, scale, x, batch):
    """Rows x (fp64 [rows][heads][dim], FP16 numbers) into codes and scale, in
    place.  batch: (start, length, table, count, rows, max_rows)."""
    start, length, table, count, rows, max_rows = batch
    for s, (first, n, at) in enumerate(spans(start, length, count, rows, max_rows)):
        met = {}
        for j in range(n):
            page = page_of(table, len(codes), s, at + j)
            if page is not None:
                met.setdefault(page, []).append((first + j, (at + j) % PAGE))
        for page, pairs in met.items():
            r, t = [p[0] for p in pairs], [p[1] for p in pairs]
            for h in range(codes.shape[1]):
                most, by, halvings = np.abs(x[r, h]).max(), scale[page, h], 0
                if not np.isfinite(x[r, h]).all():
                    by = np.nan
                elif 0 in t or by == 0:
                    by = least_scale(most)
                else:
                    while most > 127 * by:
                        by, halvings = 2 * by, halvings + 1
                if halvings:  # one rounding for all of a call's doublings
                    codes[page, h] = np.rint(codes[page, h] / 2.0 ** halvings)
                scale[page, h] = by
                codes[page, h, t] = np.rint(x[r, h] / by) if by > 0 else 0


def read(codes, scale, batch):
    start, length, table, count, rows, max_rows = batch
    out = np.full((rows, codes.shape[1], codes.shape[3]), np.nan)
    for s, (first, n, at) in enumerate(spans(start, length, count, rows, max_rows)):
        for j in range(n):
            page = page_of(table, len(codes), s, at + j)
            out[first + j] = 0 if page is None else codes[page, :, (at + j) % PAGE] * scale[page][:, None]
    return out


# ---------------------------------------------------------------- attention
def attention(kc, ks, vc, vs, q, batch, scale, window=0, causal=True):
    """(y, sum p |v|, largest |score|, sum |q||k| scale at most) per row and
    head; rows of no sequence are NaN."""
    start, length, table, count, rows, max_rows = batch
    q = np.asarray(q, np.float64)
    heads, group = kc.shape[1], q.shape[1] // kc.shape[1]
    y = np.full(q.shape, np.nan)
    size = np.zeros(q.shape)
    top = np.zeros(q.shape[:2] + (2,))
    for s, (first, n, at) in enumerate(spans(start, length, count, rows, max_rows)):
        tokens = [(t, page_of(table, len(kc), s, t)) for t in range(length[s])]
        t = np.array([t for t, p in tokens if p is not None], np.int64)
        p = np.array([p for t, p in tokens if p is not None], np.int64)
        for j in range(n):
            see = np.ones(len(t), bool)
            if causal:
                see &= t <= at + j
            if window:
                see &= t > at + j - window
            tt, pp = t[see] % PAGE, p[see]
            for h in range(q.shape[1]):
                y[first + j, h] = 0
                if not len(tt):
                    continue
                k = kc[pp, h // group, tt] * ks[pp, h // group][:, None]
                v = vc[pp, h // group, tt] * vs[pp, h // group][:, None]
                z = scale * (k @ q[first + j, h])
                w = np.exp(z - z.max())
                w /= w.sum()
                y[first + j, h] = w @ v
                size[first + j, h] = w @ np.abs(v)
                top[first + j, h] = np.abs(z).max(), (np.abs(k) @ np.abs(q[first + j, h])).max() * scale
    return y, size, top

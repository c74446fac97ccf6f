"""Inputs and checks shared by the tests of positions, cache and attention."""
import numpy as np
import torch

from oracle import kv_oracle as K
from ternary_weight_only_tern_amd import lib as L

U16, U32 = 2.0 ** -11, 2.0 ** -24
TINY16 = 2.0 ** -25  # half a step of FP16's subnormals


def dev(a, kind=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if kind is None else t.to(kind)


def half(rng, *shape, spread=1.0):
    return (spread * rng.standard_normal(shape)).astype(np.float16)


class Case:
    """A cache with contents and a batch over it, on the host and the device."""

    def __init__(self, rng, rows, lens, heads=2, dim=64, ragged=None, spare=3, extra=0, holes=(), tail=0, spread=False):
        self.rows, self.lens, self.heads, self.dim = list(rows), list(lens), heads, dim
        count = len(rows)
        need = [max(1, -(-max(n, 1) // 64)) for n in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        width = max(need) + extra
        self.table = np.full((count, width), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        for s, p, value in holes:
            self.table[s, p] = value
        ragged = len(set(rows)) > 1 if ragged is None else ragged
        self.max_rows = max(rows)
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32) if ragged else None
        self.m = sum(rows) + (tail if ragged else 0)
        self.kc = np.clip(np.rint(rng.standard_normal((pages, heads, 64, dim)) * 30), -127, 127).astype(np.int64)
        self.vc = np.clip(np.rint(rng.standard_normal((pages, heads, 64, dim)) * 30), -127, 127).astype(np.int64)
        power = rng.integers(-14, 2, (2, pages, heads)) if spread else np.full((2, pages, heads), -12)
        self.ks, self.vs = rng.integers(128, 256, (2, pages, heads)) * 2.0 ** power
        if spread:
            self.ks = self.ks * 0 + rng.integers(128, 256, (pages, heads)) * 2.0 ** -12

    @property
    def batch(self):
        return self.start, self.lens, self.table, len(self.rows), self.m, self.max_rows

    def cache(self):
        k, v = (dev(K.pack(c, keys)).view(*c.shape) for c, keys in ((self.kc, True), (self.vc, False)))
        return L.KvCache(k, v, dev(self.ks, torch.float32), dev(self.vs, torch.float32))

    def on_device(self, max_len=None):
        return L.KvBatch(dev(np.array(self.lens, np.int32)), dev(self.table), self.max_rows,
                         start=None if self.start is None else dev(self.start), max_len=max_len)


def attention_bound(y, size, top, dim, tokens, vmax):
    """The output's rounding; every weight's 11 bits (and 2^-35 of the
    reference below them, times the largest value that a span of 64 allows); a
    score's error (dim products and sums in FP32, its scale and the exponent's
    24 bits) on a weight and on the sum of weights; the sums.  An addition is
    off by a whole step at most, which the matrix instructions may take."""
    score = top[..., :1]
    error = 2 * U32 * ((dim + 8) * top[..., 1:] + 4 * score + 4)
    return U16 * np.abs(y) + TINY16 + size * (U16 + 2 * np.expm1(error) + (tokens + 64) * 2 * U32) + tokens * 2.0 ** -35 * 64 * vmax


def check_attention(c: Case, q, got, scale, window=0, causal=True, note=""):
    y, size, top = K.attention(c.kc, c.ks, c.vc, c.vs, q, c.batch, scale, window, causal)
    got = got.float().cpu().numpy().astype(np.float64)
    live = ~np.isnan(y[:, 0, 0])
    vmax = 127 * np.nanmax(c.vs) if np.size(c.vs) else 0
    bound = attention_bound(y, size, top, c.dim, max(c.lens + [1]), vmax)
    off = np.abs(got - y)[live] / bound[live]
    assert np.isfinite(got[live]).all(), f"{note}: not finite"
    assert (off <= 1).all(), f"{note}: {off.max():.3g} of the bound, {int((off > 1).sum())} values"

"""Attention where the values' scales alternate between the ends of their
documented range, and one page of larger scores leaves nothing of them."""
import numpy as np
import pytest
import torch

from kv_util import TINY16, U16, dev
from oracle import kv_oracle as K
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu

BITS = L.TERN_KV_SCALE_BITS
KERNELS = {  # rows, tiles' rows, max_len, what tern_kv_attention_parts says
    "one row": (1, 0, None, lambda n: n > 1), "one row, whole": (1, 0, 64, lambda n: n == 1), "two blocks": (20, 0, 10 ** 6, lambda n: n > 1),
    "tiles of 64": (90, 64, None, lambda n: n < -2), "tiles of 64, uncut": (90, 64, 64, lambda n: n == -2),
    "tiles of 128": (90, 128, None, lambda n: n < -2), "tiles of 128, uncut": (90, 128, 64, lambda n: n == -2),
}


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kernel", KERNELS)
def test_ends_of_the_range(kernel, dim):
    """Pages 0 and 1 have the largest and the smallest scale, scores of 0, and
    alternate 400 times; page 2 comes last with scores of 127, so that what was
    before has e^-127 = 2^-183 of it: at 2^36 against the outputs' 2^-12 and
    less, nothing.  Its tokens' scores are equal: y is the mean of its values.
    Its weights are one number, rounded to FP16 against the values and perhaps
    not in their sum (2^-11), sums of whole numbers are exact in FP32, a few
    roundings of FP32 remain (2^-20), and the output's own."""
    rows, tile, max_len, way = KERNELS[kernel]
    rng = np.random.default_rng(dim)
    kc = np.zeros((3, 1, 64, dim), np.int64)
    kc[2, 0, :, 0] = 127
    vc = rng.integers(1, 128, (3, 1, 64, dim))
    vs = np.array([[2.0 ** BITS], [2.0 ** -BITS], [2.0 ** -12]])
    cache = L.KvCache(dev(K.pack(kc, True)).view(3, 1, 64, dim), dev(K.pack(vc, False)).view(3, 1, 64, dim),
                      torch.ones((3, 1), device="cuda"), dev(vs, torch.float32))
    want = (vc[2, 0] * vs[2]).mean(axis=0)
    q = np.zeros((rows, 1, dim), np.float16)
    q[..., 0] = 1
    try:
        L.tern_kv_tile_rows(tile)
        for first in (0, 1):
            table = np.array([[first, 1 - first] * 400 + [2]], np.int32)
            batch = L.KvBatch(dev(np.array([64 * 801], np.int32)), dev(table), rows, max_len=max_len)
            parts = L.load().tern_kv_attention_parts(cache._at, L.ctypes.addressof(batch._of(cache.device, rows)), 1, 0)
            assert way(parts), parts
            got = L.tern_kv_attention(cache, batch, dev(q), scale=1.0, causal=False).double().cpu().numpy()
            assert (np.abs(got - want) <= np.abs(want) * (2 * U16 + 2.0 ** -20) + TINY16).all(), (first, got[0, 0, :4], want[:4])
    finally:
        L.tern_kv_tile_rows(0)

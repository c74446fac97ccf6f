"""What tern_kv_attention checks before it launches: these calls carry made-up
addresses, and every one of them is refused on the host, with or without a
GPU."""
import ctypes

import numpy as np
import pytest

from ternary_weight_only_tern_amd import lib as L

_held = []


def at(d):
    _held.append(d)
    return ctypes.addressof(d)


def cache(heads, dim):
    return at(L.tern_kv(heads, dim, 100, 0x10000, 0x20000, 0x30000, 0x40000))


def batch(count, max_rows, max_len):
    return at(L.tern_kv_batch(count, count * max_rows, max_rows, max_len, 4, None, 0x50000, 0x60000))


def attention(c, b, q_heads, ws, size, window=0, causal=1):
    return L.load().tern_kv_attention(c, b, 0x1000, 8, q_heads, 0.1, window, causal, 0x2000, ws, size, None)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("count,max_rows,max_len", [(1, 1, 1), (1, 1, 64), (2, 3, 100), (1, 2048, 2048), (300, 1, 2000), (1, 1, 100000), (1, 64, 4000)])
def test_a_workspace_is_aligned_whether_needed_or_not(count, max_rows, max_len, dim):
    c, b = cache(8, dim), batch(count, max_rows, max_len)
    size = L.load().tern_kv_attention_workspace_bytes(c, b, 32)
    for window, causal in ((0, 1), (0, 0), (70, 1)):
        for ws in (0x3008, 0x3001):
            assert attention(c, b, 32, ws, size, window, causal) == L.TERN_E_ALIGN


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (8, 4), (8, 8), (12, 1), (2, 40)])
def test_a_workspace_serves_every_smaller_batch(heads, group, dim):
    """Its size is looked at before its alignment, so that a refusal of the
    alignment says that the size is enough."""
    lib, c = L.load(), cache(heads, dim)
    rng = np.random.default_rng(heads * group + dim)
    for _ in range(100):
        count, max_rows, max_len = (int(2 ** rng.uniform(0, hi)) for hi in (9, 12, 17))
        size = lib.tern_kv_attention_workspace_bytes(c, batch(count, max_rows, max_len), heads * group)
        for _ in range(5):
            n = int(rng.integers(1, count + 1))
            r = int(rng.integers(1, max(1, count * max_rows // n) + 1))
            small = batch(n, r, int(rng.integers(0, max_len + 1)))
            for causal in (0, 1):
                assert attention(c, small, heads * group, 0x3008, size, 0, causal) == L.TERN_E_ALIGN, \
                    (count, max_rows, max_len, n, r, lib.tern_last_error())

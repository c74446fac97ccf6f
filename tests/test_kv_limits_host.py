"""Sizes at which a product of sizes passes 64 bits: refused on the host, with
or without a GPU (the addresses are made up)."""
import ctypes

import pytest

from ternary_weight_only_tern_amd import lib as L

_held = []


def at(d):
    _held.append(d)
    return ctypes.addressof(d)


def cache(heads, dim=64):
    return at(L.tern_kv(heads, dim, 100, 0x10000, 0x20000, 0x30000, 0x40000))


def batch(count, rows, max_rows, max_len=1000, max_pages=1):
    return at(L.tern_kv_batch(count, rows, max_rows, max_len, max_pages, 0x70000, 0x50000, 0x60000))


# workgroups: 2 x count x heads x pages that a sequence's rows may lie in, of 256 threads
# (2^29 - 63 rows lie in 2^23 pages at most)
@pytest.mark.parametrize("count,heads", [
    (1 << 29, 8),           # 2^56 workgroups, 2^64 threads
    (1 << 30, 1 << 10),     # 2^64 workgroups
    (1 << 28, 1 << 11),     # 2^63 workgroups
    ((1 << 31) - 1, 65535), (1 << 14, 64), (2, 1)])  # 2^71, 2^44, 2^25
def test_more_workgroups_than_can_be_counted(count, heads):
    lib, c, b = L.load(), cache(heads), batch(count, (1 << 29) - 63, (1 << 29) - 63)
    unsupported = L.TERN_E_UNSUPPORTED
    assert lib.tern_kv_write(c, b, 0x1000, 0, 0x2000, 0, None, None, 0, 0, None, None, None) == unsupported
    assert b"too many workgroups" in lib.tern_last_error()
    assert lib.tern_kv_read(c, b, 0x1000, 0x2000, 0, None) == unsupported
    assert b"too many workgroups" in lib.tern_last_error()

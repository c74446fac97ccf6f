"""Argument errors of rotary positions, cache and attention, their workspaces
and plans, and the frequencies, answered without a GPU."""
import ctypes

import numpy as np
import pytest

from oracle import kv_oracle as K
from ternary_weight_only_tern_amd import lib as L

INVAL, ALIGN, UNSUPPORTED, WORKSPACE = L.TERN_E_INVAL, L.TERN_E_ALIGN, L.TERN_E_UNSUPPORTED, L.TERN_E_WORKSPACE
_held = []


def at(d):
    """A descriptor's address, which stays valid."""
    _held.append(d)
    return ctypes.addressof(d)


def cache(heads=8, dim=128, pages=100, k=0x10000, v=0x20000, ks=0x30000, vs=0x40000):
    return L.tern_kv(heads, dim, pages, k, v, ks, vs)


def batch(count=2, rows=None, max_rows=3, max_len=1000, max_pages=16, start=None, len=0x50000, pages=0x60000):
    return L.tern_kv_batch(count, count * max_rows if rows is None else rows, max_rows, max_len, max_pages, start, len, pages)


def rotary(rot=128, interleaved=0, freq=0x70000, amp=1.0, eps=1e-6, norm=None):
    return L.tern_rotary(rot, interleaved, freq, amp, eps, norm)


@pytest.mark.parametrize("kw,want", [
    ({}, L.TERN_OK), (dict(dim=64), L.TERN_OK), (dict(pages=0, k=None, v=None, ks=None, vs=None), L.TERN_OK),
    (dict(heads=0), INVAL), (dict(pages=-1), INVAL), (dict(dim=96), UNSUPPORTED), (dict(dim=512), UNSUPPORTED),
    (dict(heads=70000), UNSUPPORTED), (dict(k=None), INVAL), (dict(vs=None), INVAL), (dict(k=0x10008), ALIGN),
    (dict(v=0x20004), ALIGN), (dict(ks=0x30002), ALIGN)])
def test_check(kw, want):
    c = cache(**kw)
    assert L.load().tern_kv_check(at(c)) == want


def test_null_descriptors():
    lib, c, b = L.load(), cache(), batch()
    assert lib.tern_kv_check(None) == INVAL
    assert lib.tern_kv_read(None, at(b), 16, 16, 0, None) == INVAL and lib.tern_kv_read(at(c), None, 16, 16, 0, None) == INVAL
    assert lib.tern_kv_attention_workspace_bytes(None, at(b), 8) == 0 and lib.tern_kv_attention_workspace_bytes(at(c), None, 8) == 0
    assert lib.tern_kv_attention_parts(None, at(b), 8, 0) == -1


BATCHES = [
    (dict(count=-1, rows=0), INVAL), (dict(rows=-1), INVAL), (dict(max_rows=-1), INVAL), (dict(max_len=-1), INVAL),
    (dict(max_pages=-1), INVAL), (dict(rows=7), INVAL), (dict(len=None), INVAL), (dict(pages=None), INVAL),
    (dict(len=0x50002), ALIGN), (dict(start=0x51002, rows=5), ALIGN), (dict(pages=0x60001), ALIGN),
    (dict(count=1, max_rows=(1 << 29) + 1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", BATCHES)
def test_batches(kw, want):
    lib, c, b = L.load(), cache(), batch(**kw)
    assert lib.tern_kv_read(at(c), at(b), 0x1000, 0x2000, 0, None) == want
    assert lib.tern_kv_write(at(c), at(b), 0x1000, 1024, 0x2000, 1024, None, None, 0, 0, None, None, None) == want
    assert lib.tern_kv_attention(at(c), at(b), 0x1000, 4096, 32, 0.1, 0, 1, 0x2000, 0x3000, 1 << 40, None) == want


def test_write_refusals():
    lib = L.load()

    def f(c=cache(), b=batch(), k=0x1000, ks=1024, v=0x2000, vs=1024, rope=None, q=None, qs=4096, qh=32, qr=None, qo=0x3000):
        return lib.tern_kv_write(at(c), at(b), k, ks, v, vs, rope and at(rope), q, qs, qh, qr and at(qr), qo, None)

    assert f(k=None) == INVAL and f(v=None) == INVAL and f(k=0x1008) == ALIGN
    assert f(ks=-1024) == INVAL and f(vs=1028) == ALIGN and f(ks=1) == ALIGN
    assert f(c=cache(pages=0)) == INVAL and f(c=cache(dim=80)) == UNSUPPORTED
    for r in (rotary(rot=130), rotary(rot=-2), rotary(rot=3), rotary(freq=None)):
        assert f(rope=r) == INVAL and f(q=0x4000, qr=r) == INVAL
    assert f(rope=rotary(freq=0x70004)) == ALIGN and f(rope=rotary(norm=0x80008)) == ALIGN
    assert f(q=0x4000) == INVAL and b"q_rope" in lib.tern_last_error()
    assert f(q=0x4000, qr=rotary(), qo=None) == INVAL and f(q=0x4000, qr=rotary(), qh=-1) == INVAL
    assert f(q=0x4008, qr=rotary()) == ALIGN and f(q=0x4000, qr=rotary(), qo=0x3008) == ALIGN
    assert f(q=0x4000, qr=rotary(), qs=4100) == ALIGN
    assert f(q=0x4000, qr=rotary(), qo=0x4000, qs=4104) == INVAL and b"q_out is q" in lib.tern_last_error()
    empty = batch(count=0, len=None, pages=None)
    assert f(b=empty, k=None, v=None) == L.TERN_OK and f(b=batch(max_rows=0), k=None, v=None) == L.TERN_OK
    assert f(b=batch(count=1 << 20, max_rows=500)) == UNSUPPORTED and b"too many workgroups" in lib.tern_last_error()


def test_read_refusals():
    lib, c, b = L.load(), cache(), batch()
    assert lib.tern_kv_read(at(c), at(b), 0x1000, 0x2000, 2, None) == UNSUPPORTED
    assert lib.tern_kv_read(at(c), at(b), 0x1008, 0x2000, 0, None) == ALIGN and lib.tern_kv_read(at(c), at(b), None, 0x2004, 1, None) == ALIGN
    assert lib.tern_kv_read(at(c), at(b), None, None, 0, None) == L.TERN_OK
    assert lib.tern_kv_read(at(c), at(batch(count=0)), 1, 1, 0, None) == L.TERN_OK


def test_attention_refusals():
    lib = L.load()

    def f(c=cache(), b=batch(max_len=100000), q=0x1000, qs=4096, heads=32, scale=0.1, window=0, causal=1, y=0x2000, ws=0x3000, nb=1 << 40):
        return lib.tern_kv_attention(at(c), at(b), q, qs, heads, scale, window, causal, y, ws, nb, None)

    assert f(q=None) == INVAL and f(y=None) == INVAL and f(q=0x1004) == ALIGN and f(y=0x2008) == ALIGN and f(ws=0x3008) == ALIGN
    assert f(heads=0) == INVAL and f(heads=12) == INVAL and f(heads=80000 // 8 * 8) == UNSUPPORTED
    assert f(scale=-1.0) == INVAL and f(scale=float("nan")) == INVAL and f(scale=float("inf")) == INVAL
    assert f(window=-1) == INVAL and f(window=5, causal=0) == UNSUPPORTED
    assert f(qs=4097) == ALIGN and f(qs=-8) == INVAL and f(qs=(1 << 23) + 8) == UNSUPPORTED
    assert f(c=cache(pages=0)) == INVAL
    assert f(b=batch(count=1 << 22)) == UNSUPPORTED and f(b=batch(count=1 << 12, max_pages=1 << 20)) == UNSUPPORTED
    assert f(b=batch(count=1, max_rows=1 << 28), heads=64) == UNSUPPORTED
    need = lib.tern_kv_attention_workspace_bytes(at(cache()), at(batch(max_len=100000)), 32)
    assert need > 256 and f(nb=0) == WORKSPACE and f(ws=None) == WORKSPACE
    assert f(b=batch(count=0, len=None, pages=None), q=None, y=None, ws=None, nb=0) == L.TERN_OK


def test_rope_refusals():
    lib = L.load()

    def f(r=rotary(rot=64), x=0x1000, xs=640, m=3, heads=5, dim=128, pos=0x2000, out=0x3000, os=640):
        return lib.tern_rope(x, xs, m, heads, dim, pos, r and at(r), out, os, None)

    assert f(m=-1) == INVAL and f(heads=-1) == INVAL and f(dim=-8) == INVAL and f(r=None) == INVAL
    assert f(dim=100) == UNSUPPORTED and f(dim=520) == UNSUPPORTED
    assert f(x=None) == INVAL and f(out=None) == INVAL and f(pos=None) == INVAL
    assert f(x=0x1002) == ALIGN and f(xs=636) == ALIGN and f(os=641) == ALIGN and f(pos=0x2002) == ALIGN
    assert f(r=rotary(rot=136)) == INVAL and f(r=rotary(rot=7)) == INVAL and f(r=rotary(rot=64, norm=0x4004)) == ALIGN
    assert f(os=632) == INVAL and f(os=0) == INVAL  # rows of out that overlap
    assert f(out=0x1000, os=648) == INVAL and f(out=0x1000, xs=1280) == INVAL  # in place at another stride
    for kw in (dict(m=0), dict(heads=0), dict(dim=0)):
        assert f(x=None, out=None, pos=None, **kw) == L.TERN_OK


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 1), (8, 4), (8, 8), (12, 1), (2, 40)])
def test_a_workspace_serves_every_smaller_batch(heads, group, dim):
    """It is checked before its alignment; sizes do not grow without end."""
    lib, c = L.load(), cache(heads=heads, dim=dim)
    rng = np.random.default_rng(heads * group + dim)
    for _ in range(300):
        count, max_rows, max_len = (int(2 ** rng.uniform(0, hi)) for hi in (9, 12, 17))
        big = batch(count=count, max_rows=max_rows, max_len=max_len, max_pages=4)
        size = lib.tern_kv_attention_workspace_bytes(at(c), at(big), heads * group)
        assert 256 <= size <= (4096 * 32 * 2 * (dim + 2) * 4) + count * heads * 8
        for _ in range(5):
            n = int(rng.integers(1, count + 1))
            r = int(rng.integers(1, max(1, count * max_rows // n) + 1))
            small = batch(count=n, max_rows=r, max_len=int(rng.integers(0, max_len + 1)), max_pages=4)
            assert lib.tern_kv_attention(at(c), at(small), 0x1000, 8, heads * group, 0.1, 0, 1, 0x2000, 0x3008, size, None) in (ALIGN, L.TERN_E_HIP), \
                (count, max_rows, max_len, n, r, small.max_len, lib.tern_last_error())


def test_which_way_a_call_goes():
    lib, c = L.load(), cache()
    parts = lambda q_heads=32, c=c, window=0, **kw: lib.tern_kv_attention_parts(at(c), at(batch(**kw)), q_heads, window)
    assert parts(count=1, max_rows=1, max_len=4001) == 504 and parts(count=64, max_rows=1, max_len=8192) == 2048
    assert parts(count=1, max_rows=1, max_len=100) == 8  # whole units
    assert parts(count=4, max_rows=5, max_len=120000) == 1024  # two blocks of rows
    assert parts(count=1, max_rows=9, max_len=5000) < -2 and parts(count=1, max_rows=2048, max_len=4000) == -2
    assert parts(count=1, max_rows=4, max_len=5000, c=cache(dim=256)) == 632 and parts(count=1, max_rows=8, max_len=5000, c=cache(dim=256)) < -2
    assert parts(count=8, max_rows=8, max_len=4097) == 1024 and parts(count=8, max_rows=8, max_len=4096) < -2  # 4160, 4096 pages
    assert parts(count=1, max_rows=1, max_len=100000, window=100) == 8 and parts(count=0) == 0  # three pages are not cut
    assert parts(count=1, max_rows=1, max_len=100000, window=300) == 8 and parts(count=1, max_rows=1, max_len=100000, window=1200) == 160
    assert parts(count=64, max_rows=1, max_len=3008) == 512 and parts(count=64, max_rows=1, max_len=3200) == 2048  # 12 pages a wavefront
    assert parts(count=256, max_rows=1, max_len=2048) == 2048 and parts(count=300, max_rows=1, max_len=2400) == 2048  # 64 units a page
    assert parts(count=300, max_rows=1, max_len=2368) == 2400
    # tiles: no more parts than pay for their joining
    assert parts(count=1, max_rows=512, max_len=512) == -2 and parts(count=1, max_rows=512, max_len=8000) == -5
    assert parts(count=64, max_rows=512, max_len=8000) == -2 and parts(count=1, max_rows=64, max_len=4000) == -17
    assert parts(count=1, max_rows=64, max_len=100000, window=64) == -2  # three pages
    assert parts(q_heads=30) == -1 and parts(window=-1) == -1


def test_rows_of_tiles():
    lib, c = L.load(), cache()
    parts = lambda **kw: lib.tern_kv_attention_parts(at(c), at(batch(**kw)), 32, 0)
    big = batch(count=1, max_rows=512, max_len=8000)
    size = lib.tern_kv_attention_workspace_bytes(at(c), at(big), 32)
    assert L.tern_kv_tile_rows() == 0 and parts(count=1, max_rows=64, max_len=4000) == -17
    try:
        assert L.tern_kv_tile_rows(64) == 0 and L.tern_kv_tile_rows(96) == 64
        assert parts(count=1, max_rows=512, max_len=8000) == -3
        assert lib.tern_kv_attention_workspace_bytes(at(c), at(big), 32) == size
        assert L.tern_kv_tile_rows(128) == 64 and parts(count=1, max_rows=512, max_len=8000) == -5
    finally:
        assert L.tern_kv_tile_rows(0) in (64, 128)


def test_frequencies():
    for kind, name in ((L.TERN_ROPE_PLAIN, "plain"), (L.TERN_ROPE_LINEAR, "linear"), (L.TERN_ROPE_BASE, "base"),
                       (L.TERN_ROPE_RAMP, "ramp"), (L.TERN_ROPE_WAVES, "waves")):
        for rot, base, factor in ((128, 1e6, 4.0), (64, 1e4, 32.0), (2, 500.0, 2.0), (90, 1e4, 1.0)):
            got, amp = L.tern_rope_frequencies(rot, base, kind, factor, 1.0, 32.0, 4096)
            want, top = K.frequencies(rot, base, name, factor)
            assert np.allclose(got.numpy(), want, rtol=1e-13, atol=0) and np.float32(top) == np.float32(amp), (name, rot)
    assert L.tern_rope_frequencies(0)[0].numel() == 0


@pytest.mark.parametrize("kw,want", [
    (dict(rot=3), INVAL), (dict(rot=64, base=1.0), INVAL), (dict(rot=64, base=float("inf")), INVAL), (dict(rot=64, scaling=5), UNSUPPORTED),
    (dict(rot=64, scaling=L.TERN_ROPE_LINEAR, factor=0.5), INVAL), (dict(rot=64, scaling=L.TERN_ROPE_RAMP, low=4.0, high=4.0), INVAL),
    (dict(rot=64, scaling=L.TERN_ROPE_WAVES, factor=2.0, trained=0), INVAL), (dict(rot=-2), INVAL)])
def test_frequency_refusals(kw, want):
    with pytest.raises(L.TernError) as e:
        L.tern_rope_frequencies(**kw)
    assert e.value.status == want


def test_binding_refuses_what_is_not_on_a_gpu():
    import torch
    with pytest.raises(ValueError):
        L.Rope(torch.zeros(4, dtype=torch.float64))
    with pytest.raises(ValueError):
        L.KvCache(*(torch.zeros(1),) * 4)
    with pytest.raises(ValueError):
        L.KvBatch(torch.zeros(2, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32), 1)

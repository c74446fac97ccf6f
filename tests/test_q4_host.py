"""Argument errors of the 4-bit layers' C ABI, answered without a GPU."""
import ctypes

import pytest

from ternary_weight_only_tern_amd import lib as L

P = ctypes.c_void_p


def q4(n=64, k=256, group=64, count=1, codes=0x10000, scale=0x20000, zero=None):
    return L.tern_q4(n, k, group, count, codes, scale, zero)


def at(d):
    return ctypes.addressof(d)


@pytest.mark.parametrize("kw,want", [
    ({}, L.TERN_OK), (dict(group=32), L.TERN_OK), (dict(k=0, codes=None, scale=None), L.TERN_OK),
    (dict(n=0, codes=None, scale=None), L.TERN_OK),
    (dict(n=-1), L.TERN_E_INVAL), (dict(k=-64), L.TERN_E_INVAL), (dict(count=-1), L.TERN_E_INVAL),
    (dict(group=16), L.TERN_E_UNSUPPORTED), (dict(group=96), L.TERN_E_UNSUPPORTED), (dict(group=0), L.TERN_E_UNSUPPORTED),
    (dict(group=256), L.TERN_E_UNSUPPORTED), (dict(k=96), L.TERN_E_UNSUPPORTED), (dict(n=0x7fffffff), L.TERN_E_UNSUPPORTED), (dict(k=(1 << 22) + 64), L.TERN_E_UNSUPPORTED),
    (dict(codes=None), L.TERN_E_INVAL), (dict(scale=None), L.TERN_E_INVAL),
    (dict(codes=0x10008), L.TERN_E_ALIGN), (dict(scale=0x20001), L.TERN_E_ALIGN)])
def test_check(kw, want):
    d = q4(**kw)
    assert L.load().tern_q4_check(at(d)) == want


def test_null_descriptor():
    lib = L.load()
    assert lib.tern_q4_check(None) == L.TERN_E_INVAL
    assert lib.tern_q4_workspace_bytes(None, 1) == 0
    assert lib.tern_route(P(16), 0, 1, None, P(16), P(16), None) == L.TERN_E_INVAL


def test_gemm_refusals():
    lib = L.load()
    d = q4(n=64, k=4096)
    g = lambda x=0x1000, m=1, y=0x2000, dt=0, ws=0x3000, nb=1 << 30, d=d: lib.tern_q4_gemm(at(d), x, m, y, dt, ws, nb, None)
    assert g(m=-1) == L.TERN_E_INVAL
    assert g(x=None) == L.TERN_E_INVAL and g(y=None) == L.TERN_E_INVAL
    assert g(x=0x1008) == L.TERN_E_ALIGN and g(y=0x2001) == L.TERN_E_ALIGN and g(y=0x2002, dt=1) == L.TERN_E_ALIGN
    assert g(dt=2) == L.TERN_E_UNSUPPORTED
    assert g(d=q4(count=2)) == L.TERN_E_INVAL
    assert g(m=0, x=None, y=None) == L.TERN_OK
    assert g(d=q4(n=0), x=None, y=None) == L.TERN_OK
    need = lib.tern_q4_workspace_bytes(at(d), 400)
    assert need > 256
    assert g(m=400, nb=need - 1) == L.TERN_E_WORKSPACE and g(m=400, ws=None) == L.TERN_E_WORKSPACE
    assert g(m=400, ws=0x3008) == L.TERN_E_ALIGN


def test_pack_refusals():
    lib = L.load()
    d = q4()
    assert lib.tern_q4_pack(None, at(d), 0x1000, 256, None) == L.TERN_E_INVAL
    assert lib.tern_q4_pack(0x1004, at(d), 0x1000, 256, None) == L.TERN_E_ALIGN
    assert lib.tern_q4_pack(0x1000, at(d), None, 0, None) == L.TERN_E_WORKSPACE
    assert lib.tern_q4_unpack(at(d), None, None) == L.TERN_E_INVAL
    empty = q4(n=0)
    assert lib.tern_q4_unpack(at(empty), None, None) == L.TERN_OK


ROUTER = dict(experts=64, topk=8, score=1, groups=8, group_best=2, keep_groups=4, renorm=1, scale=1.0, bias=None)


@pytest.mark.parametrize("kw,want", [
    (dict(experts=0), L.TERN_E_INVAL), (dict(experts=60), L.TERN_E_INVAL), (dict(groups=0), L.TERN_E_INVAL),
    (dict(experts=2048), L.TERN_E_UNSUPPORTED), (dict(experts=256, groups=128), L.TERN_E_UNSUPPORTED),
    (dict(keep_groups=0), L.TERN_E_INVAL), (dict(keep_groups=9), L.TERN_E_INVAL),
    (dict(group_best=0), L.TERN_E_UNSUPPORTED), (dict(group_best=3), L.TERN_E_UNSUPPORTED),
    (dict(topk=0), L.TERN_E_INVAL), (dict(topk=33), L.TERN_E_INVAL), (dict(score=2), L.TERN_E_UNSUPPORTED),
    (dict(experts=1024, topk=65), L.TERN_E_UNSUPPORTED), (dict(bias=0x1002), L.TERN_E_ALIGN)])
def test_route_refusals(kw, want):
    r = L.tern_router(**{**ROUTER, **kw})
    assert L.load().tern_route(0x1000, 1, 4, at(r), 0x2000, 0x3000, None) == want


def test_route_pointers():
    lib = L.load()
    r = L.tern_router(**ROUTER)
    f = lambda l=0x1000, dt=1, m=4, ids=0x2000, w=0x3000: lib.tern_route(l, dt, m, at(r), ids, w, None)
    assert f(l=None) == L.TERN_E_INVAL and f(ids=None) == L.TERN_E_INVAL and f(w=None) == L.TERN_E_INVAL
    assert f(l=0x1002) == L.TERN_E_ALIGN and f(ids=0x2002) == L.TERN_E_ALIGN and f(dt=5) == L.TERN_E_UNSUPPORTED
    assert f(m=-1) == L.TERN_E_INVAL and f(m=0, l=None) == L.TERN_OK


def test_experts_refusals():
    lib = L.load()
    up, down = q4(n=128, k=256, count=4), q4(n=96, k=64, count=4)
    need = lib.tern_q4_experts_workspace_bytes(at(up), at(down), 10, 2)
    assert need > 0

    def f(up=up, down=down, x=0x1000, m=10, ids=0x2000, w=0x3000, topk=2, y=0x4000, dt=0, ws=0x5000, nb=need):
        return lib.tern_q4_experts(at(up), at(down), x, m, ids, w, topk, y, dt, ws, nb, None)

    assert f(m=-1) == L.TERN_E_INVAL and f(topk=0) == L.TERN_E_INVAL
    assert f(up=q4(n=128, k=256, count=5)) == L.TERN_E_INVAL
    assert f(up=q4(n=130, k=256, count=4)) == L.TERN_E_INVAL and f(up=q4(n=129, k=256, count=4)) == L.TERN_E_INVAL
    assert f(up=q4(n=128, count=0), down=q4(k=64, count=0)) == L.TERN_E_INVAL
    assert f(up=q4(n=128, count=2000), down=q4(k=64, count=2000)) == L.TERN_E_UNSUPPORTED
    assert f(m=1 << 30, topk=2) == L.TERN_E_UNSUPPORTED and f(m=1, topk=(1 << 19) + 1) == L.TERN_E_UNSUPPORTED
    for kw in (dict(x=None), dict(ids=None), dict(w=None), dict(y=None)):
        assert f(**kw) == L.TERN_E_INVAL
    assert f(x=0x1008) == L.TERN_E_ALIGN and f(ids=0x2002) == L.TERN_E_ALIGN and f(ws=0x5008) == L.TERN_E_ALIGN
    assert f(dt=9) == L.TERN_E_UNSUPPORTED and f(nb=need - 1) == L.TERN_E_WORKSPACE and f(ws=None) == L.TERN_E_WORKSPACE
    assert f(m=0, x=None, ids=None, w=None, y=None, ws=None, nb=0) == L.TERN_OK


def test_grids_past_32_bits_are_refused():
    """Sizes whose product would need more threads than a launch counts are
    refused before anything is launched."""
    lib = L.load()

    def g(m, n, k):
        d = q4(n=n, k=k)
        return lib.tern_q4_gemm(at(d), 0x1000, m, 0x2000, 0, 0x3000, 1 << 62, None)

    assert g(0x7fffffff, 16, 64) == L.TERN_E_UNSUPPORTED and b"too large" in lib.tern_last_error()
    for m, n, k in ((0x7fffff00, 16, 64), (1 << 20, 1 << 20, 64), (1, 0x7fffff00, 64), (9, 0x7fffff00, 64), (160, 0x7fffff00, 64)):
        assert g(m, n, k) == L.TERN_E_UNSUPPORTED and b"too many workgroups" in lib.tern_last_error(), (m, n, k)

    def e(m, n, count):
        up, down = q4(n=64, k=64, group=32, count=count), q4(n=n, k=32, group=32, count=count)
        return lib.tern_q4_experts(at(up), at(down), 0x1000, m, 0x2000, 0x3000, 1, 0x4000, 0, 0x5000, 1 << 62, None)

    assert e(1 << 15, 1 << 22, 1024) == L.TERN_E_UNSUPPORTED and b"too many workgroups" in lib.tern_last_error()
    assert e(1, 1 << 27, 8) == L.TERN_E_UNSUPPORTED


def test_sizes_past_32_bits_are_refused():
    assert L._count(2 ** 31 - 1) == 2 ** 31 - 1
    with pytest.raises(ValueError):
        L._count(2 ** 31)


@pytest.mark.parametrize("m,topk,count,n", [
    (1, 1, 8, 1 << 26), (16, 1, 1, 1 << 27), (32, 1, 2, 1 << 27), (2, 16, 1, 1 << 27), (400, 1, 1024, 1 << 30),
    (1 << 15, 1, 64, 1 << 24)])
def test_experts_grids_are_checked_before_any_launch(m, topk, count, n):
    """A down product that needs too large a grid is refused before the gate
    and up product runs: slot by slot (however few experts share the slots)
    and on tiles."""
    lib = L.load()
    up, down = q4(n=64, k=64, group=32, count=count), q4(n=n, k=32, group=32, count=count)
    need = lib.tern_q4_experts_workspace_bytes(at(up), at(down), m, topk)
    got = lib.tern_q4_experts(at(up), at(down), 0x1000, m, 0x2000, 0x3000, topk, 0x4000, 0, 0x5000, need, None)
    assert got == L.TERN_E_UNSUPPORTED
    assert lib.tern_last_error().startswith(b"m=%d, n=" % m), lib.tern_last_error()


@pytest.mark.parametrize("hidden,inner,count,topk", [(7168, 2048, 256, 8), (4096, 2048, 64, 8), (65536, 32, 4, 1)])
def test_experts_workspace_does_not_grow_without_end(hidden, inner, count, topk):
    """Tokens are taken in rounds of about 1 GiB of partials and inner values."""
    lib = L.load()
    up, down = q4(n=2 * inner, k=512, count=count), q4(n=hidden, k=inner, group=32, count=count)
    sizes = [lib.tern_q4_experts_workspace_bytes(at(up), at(down), m, topk) for m in (65536, 1 << 17, 1 << 20)]
    assert 1 << 29 < min(sizes) and max(sizes) <= (1 << 30) + (1 << 24), sizes


@pytest.mark.parametrize("n,k,group", [(4096, 4096, 128), (64, 4096, 64), (1000, 9728, 32), (12288, 4096, 128), (33, 128, 64)])
def test_gemm_workspace_grows_with_the_rows(n, k, group):
    """A workspace for some rows serves every call with fewer."""
    lib = L.load()
    d = q4(n=n, k=k, group=group)
    rows = [*range(1, 700), 1023, 1024, 1025, 4096, 20000]
    sizes = [lib.tern_q4_workspace_bytes(at(d), m) for m in rows]
    assert sizes == sorted(sizes)
    assert sizes[0] == 256 and (sizes[-1] > 256) == (k > 2048 and n < 12288)  # K parts: long rows, few tiles


@pytest.mark.parametrize("hidden,inner,count,topk", [(4096, 14336, 8, 2), (2560, 1024, 64, 8), (64, 32, 4, 1), (60000, 32, 3, 40), (4096, 2048, 1, 2)])
def test_experts_workspace_grows_with_the_tokens(hidden, inner, count, topk):
    lib = L.load()
    up, down = q4(n=2 * inner, k=512, count=count), q4(n=hidden, k=inner, group=32, count=count)
    rows = [*range(1, 900), 2047, 2048, 2049, 5000, 20000, 65536, 1 << 17]
    sizes = [lib.tern_q4_experts_workspace_bytes(at(up), at(down), m, topk) for m in rows]
    assert sizes == sorted(sizes)
    for m, size in zip(rows, sizes):  # each is enough, and checked before the workspace's alignment
        call = lambda nb: lib.tern_q4_experts(at(up), at(down), 0x1000, m, 0x2000, 0x3000, topk, 0x4000, 0, 0x5008, nb, None)
        assert call(size) == L.TERN_E_ALIGN and call(255) == L.TERN_E_WORKSPACE


def test_workspaces_of_refused_sizes_are_refused():
    """The binding makes no workspace for a call that would be refused."""
    from types import SimpleNamespace
    descs = [q4(n=64, k=256), q4(n=128, k=256, count=4), q4(n=96, k=64, count=4)]
    w, up, down = (SimpleNamespace(_at=at(d), device="cpu") for d in descs)
    assert L.tern_q4_workspace(w, 0).numel() == 256 and L.tern_q4_experts_workspace(up, down, 0, 2).numel() >= 256
    assert L.tern_q4_experts_workspace(up, down, 100, 2).numel() > 256
    for m in (-1, 0x7fffffff, 1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError):
            L.tern_q4_workspace(w, m)
    for u, d, m, topk in ((up, down, -1, 2), (up, down, 10, 0), (up, up, 10, 2), (up, down, 1 << 30, 2), (up, down, 1 << 32, 2),
                          (up, down, 10, (1 << 32) + 2)):
        with pytest.raises(ValueError):
            L.tern_q4_experts_workspace(u, d, m, topk)


def test_kernels_a_call_takes():
    """The tiles of the products and of the experts, and -1 for what is refused."""
    lib = L.load()
    w = q4(n=12288, k=4096, group=128)
    assert [lib.tern_q4_tile_rows(at(w), m) for m in (0, 1, 16, 160, 400, 512)] == [0, 0, 0, 0, 96, 64]
    tall = q4(n=131072, k=2560, group=128)
    assert [lib.tern_q4_tile_rows(at(tall), m) for m in (1, 24, 2048)] == [0, 32, 128]
    assert lib.tern_q4_tile_rows(at(w), -1) == -1 and lib.tern_q4_tile_rows(None, 1) == -1
    up, down = q4(n=2048, k=2560, group=128, count=64), q4(n=2560, k=1024, group=128, count=64)
    rows = [lib.tern_q4_experts_tile_rows(at(up), at(down), m, 8) for m in (1, 4, 8, 41, 100, 2048)]
    assert rows == [0, 0, 8, 16, 32, 64]
    assert lib.tern_q4_experts_tile_rows(at(up), at(up), 1, 8) == -1


def test_matrices_past_the_tiles_buffers_stay_on_the_rows_kernel():
    """The tile kernel holds a matrix's scales in one buffer below 2 GiB at
    the shortest groups."""
    lib = L.load()
    for n, k, rows in ((1 << 20, 32640, 128), (1 << 20, 32768, 0), ((1 << 20) + 64, 32768, 0)):
        w = q4(n=n, k=k, group=128)
        assert lib.tern_q4_tile_rows(at(w), 2048) == rows
    for inner, width, want in ((1 << 20, 16, 64), (1 << 20, 32736, 64), (1 << 20, 32768, 16), (1 << 14, 1 << 20, 64), (1 << 15, 1 << 20, 16)):
        up, down = q4(n=2 * inner, k=512, group=128), q4(n=width, k=inner, group=128)
        assert lib.tern_q4_experts_tile_rows(at(up), at(down), 100, 1) == want, (inner, width)


@pytest.mark.parametrize("hidden,inner,count,topk,most", [(2560, 1024, 64, 8, 4), (4096, 14336, 8, 2, 1), (4096, 2048, 8, 2, 4), (1024, 512, 4, 1, 32),
                                                          (65536, 65536, 1, 1, 1), (64, 64, 1024, 16, 2)])
def test_few_slots_that_share_experts_go_to_tiles(hidden, inner, count, topk, most):
    """Up to `most` tokens slot by slot; from there on what would be read again
    counts for more than the launches that sorting costs."""
    lib = L.load()
    up, down = q4(n=2 * inner, k=hidden, group=64, count=count), q4(n=hidden, k=inner, group=64, count=count)
    rows = [lib.tern_q4_experts_tile_rows(at(up), at(down), m, topk) for m in range(1, 50)]
    assert not any(rows[:most]) and all(rows[most:]), rows

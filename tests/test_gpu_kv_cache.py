"""tern_kv_write and tern_kv_read on the GPU: bytes and scales equal to the
oracle's, whose rounding is exact."""
import numpy as np
import pytest
import torch

from gpu_util import say
from kv_util import Case, dev, half
from oracle import kv_oracle as K
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu

NAN16 = np.float16(np.nan)


def check_cache(c, cache, note=""):
    """Every scale, and every byte, also those that no row wrote."""
    for name, codes, scale, got, by in (("k", c.kc, c.ks, cache.k, cache.k_scale), ("v", c.vc, c.vs, cache.v, cache.v_scale)):
        assert np.array_equal(by.cpu().numpy().astype(np.float64), scale, equal_nan=True), f"{note}: scales of {name}"
        raw = got.cpu().numpy().reshape(*codes.shape[:2], -1)
        wrong = K.unpack(raw, c.dim, name == "k") != codes
        assert not wrong.any(), f"{note}: {int(wrong.sum())} codes of {name}, first at {np.argwhere(wrong)[0]}"


def write(c, k, v, **kw):
    cache = kw.pop("cache", None) or c.cache()
    L.tern_kv_write(cache, c.on_device(), dev(k), dev(v), **kw)
    K.write(c.kc, c.ks, k.astype(np.float64), c.batch)
    K.write(c.vc, c.vs, v.astype(np.float64), c.batch)
    return cache


CASES = [
    # rows, lens
    ([1], [1]), ([1], [64]), ([1], [65]), ([1, 1, 1], [5, 128, 63]), ([64], [64]), ([65], [65]), ([63], [127]), ([2], [65]),
    ([66], [129]), ([130, 1, 17], [200, 64, 17]), ([3, 3], [2, 0]), ([5, 9], [3, 70]), ([1, 0, 4], [9, 50, 64]), ([300], [333]),
]


@pytest.mark.parametrize("heads,dim", [(1, 64), (3, 128), (2, 256)])
@pytest.mark.parametrize("rows,lens", CASES)
def test_write_and_read(rows, lens, heads, dim):
    say("kv write", rows, lens, heads, dim)
    rng = np.random.default_rng(sum(rows) + sum(lens) + dim)
    c = Case(rng, rows, lens, heads, dim, tail=2)
    k, v = half(rng, c.m, heads, dim), half(rng, c.m, heads, dim, spread=20.0)  # v grows, k mostly does not
    cache = write(c, k, v)
    check_cache(c, cache)
    again = write(c, k, v, cache=cache)  # the same rows again: nothing grows, nothing changes
    check_cache(c, again, "again")
    for kind, step in ((L.TERN_F16, np.float16), (L.TERN_F32, np.float32)):
        kind_t = torch.float16 if kind == L.TERN_F16 else torch.float32
        out = [torch.full((c.m, heads, dim), 77.0, dtype=kind_t, device="cuda") for _ in range(2)]
        L.tern_kv_read(cache, c.on_device(), k=out[0], v=out[1])
        for got, codes, scale in ((out[0], c.kc, c.ks), (out[1], c.vc, c.vs)):
            want = K.read(codes, scale, c.batch)
            want[np.isnan(want)] = 77  # rows of no sequence stay as they were
            with np.errstate(over="ignore"):
                assert np.array_equal(got.cpu().numpy(), want.astype(step))
    got = L.tern_kv_read(cache, c.on_device(), rows=c.m, y_dtype=L.TERN_F32)
    assert got[0].dtype == torch.float32 and got[0].shape == (c.m, heads, dim)


def test_token_by_token_errors_stay_below_a_step():
    """A page filled a token at a time, growing on the way: the scale doubles
    from the first token's, every value within a step of its last scale."""
    rng = np.random.default_rng(3)
    c = Case(rng, [1], [1], heads=2, dim=128)
    c.table[0, 0] = 1
    cache = c.cache()
    rows = half(rng, 64, 2, 128) * np.exp2(np.arange(64) / 12).astype(np.float16)[:, None, None]
    for t in range(64):
        c.lens = [t + 1]
        write(c, rows[t:t + 1], rows[t:t + 1], cache=cache)
        check_cache(c, cache, f"token {t}")
    back = c.kc[1].transpose(1, 0, 2) * c.ks[1][None, :, None]
    assert (np.abs(back - rows) < c.ks[1][None, :, None]).all()
    assert (c.ks[1] > 8 * np.array([K.least_scale(m) for m in np.abs(rows[0]).max(axis=-1)])).all()


@pytest.mark.parametrize("spread", [2.0 ** -24, 1e-5, 1e-2, 1e4])
def test_sizes_of_values(spread):
    """From subnormals to FP16's largest, and ties: multiples of half a step."""
    rng = np.random.default_rng(13)
    c = Case(rng, [70, 64], [70, 90], heads=2, dim=64)
    k = np.clip(half(rng, c.m, 2, 64, spread=1.0).astype(np.float64) * spread, -65504, 65504).astype(np.float16)
    v = (rng.integers(-254, 255, (c.m, 2, 64)) * 0.5).astype(np.float16)
    v[:, :, 0] = 127
    cache = write(c, k, v)
    check_cache(c, cache)


def test_zeros_and_pages_of_zeros():
    """A page of zeros has scale 0 and takes a scale with the first value."""
    rng = np.random.default_rng(17)
    c = Case(rng, [3], [3], heads=2, dim=64)
    cache = write(c, np.zeros((3, 2, 64), np.float16), np.zeros((3, 2, 64), np.float16))
    check_cache(c, cache)
    assert (c.ks[c.table[0, 0]] == 0).all()
    c.rows, c.max_rows, c.lens, c.m = [2], 2, [5], 2
    cache = write(c, half(rng, 2, 2, 64), half(rng, 2, 2, 64), cache=cache)
    check_cache(c, cache)


def test_infinities_poison_their_page_and_head_alone():
    rng = np.random.default_rng(19)
    c = Case(rng, [70, 1], [70, 30], heads=3, dim=64)
    k, v = half(rng, c.m, 3, 64), half(rng, c.m, 3, 64)
    k[5, 1, 9], v[66, 0, 3], v[70, 2, 63] = np.nan, -np.inf, np.inf
    cache = write(c, k, v)
    check_cache(c, cache)
    assert np.isnan(c.ks[c.table[0, 0], 1]) and np.isnan(c.vs[c.table[0, 1], 0]) and np.isnan(c.vs[c.table[1, 0], 2])
    assert int(np.isnan(c.ks).sum()) == 1 and int(np.isnan(c.vs).sum()) == 2
    back = L.tern_kv_read(cache, c.on_device(), rows=c.m)[0]
    assert torch.isnan(back[:64, 1]).all() and torch.isfinite(back[:, 0]).all() and torch.isfinite(back[64:70]).all()
    c.rows, c.max_rows, c.lens, c.m, c.start = [1, 1], 1, [65, 31], 2, None  # the pages' first token, and a later one
    cache = write(c, half(rng, 2, 3, 64), half(rng, 2, 3, 64), cache=cache)
    check_cache(c, cache, "after")
    assert np.isfinite(c.vs[c.table[0, 1], 0]) and np.isnan(c.vs[c.table[1, 0], 2])


def test_pages_that_are_not_there():
    """Numbers outside the cache and tokens behind the table: not written,
    read as zeros."""
    rng = np.random.default_rng(23)
    c = Case(rng, [200, 20], [260, 40], heads=2, dim=64, holes=[(0, 1, -1), (0, 2, 10 ** 6), (1, 0, -(2 ** 31))])
    c.lens[0] = 64 * c.table.shape[1] + 30  # its last rows lie behind the table
    cache = write(c, half(rng, c.m, 2, 64), half(rng, c.m, 2, 64))
    check_cache(c, cache)
    got = L.tern_kv_read(cache, c.on_device(), rows=c.m, y_dtype=L.TERN_F32)
    for g, codes, scale in ((got[0], c.kc, c.ks), (got[1], c.vc, c.vs)):
        want = K.read(codes, scale, c.batch)
        assert np.array_equal(g.cpu().numpy(), want)


def test_garbage_in_scales_ends():
    """Scales that nobody wrote (negative, infinite, tiny): the call ends, the
    page of another token is right."""
    rng = np.random.default_rng(29)
    c = Case(rng, [1, 1, 1, 1], [7, 8, 9, 1], heads=1, dim=64)
    cache = c.cache()
    for s, bad in enumerate((-3.0, np.inf, 1e-45)):
        cache.k_scale[int(c.table[s, 0])] = bad
    L.tern_kv_write(cache, c.on_device(), dev(half(rng, 4, 1, 64)), dev(half(rng, 4, 1, 64)))
    torch.cuda.synchronize()
    assert torch.isfinite(cache.k_scale[int(c.table[3, 0])]).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot,normed", [(64, 64, False), (128, 128, True), (128, 64, True), (256, 90, False), (256, 256, True), (128, 0, True)])
def test_write_turns_as_tern_rope(dim, rot, normed, interleaved):
    """k turned in the write gives the bytes that tern_rope's rows give, q
    turned beside it tern_rope's rows."""
    say("kv write rope", dim, rot, normed, interleaved)
    rng = np.random.default_rng(dim + rot)
    c = Case(rng, [70, 3, 1], [300, 2, 64], heads=2, dim=dim)
    freq, _ = K.frequencies(rot, 1e4)
    kr, qr = (L.Rope(dev(freq), interleaved, 1.1, dev(half(rng, dim)) if normed else None) for _ in range(2))
    fused = dev(half(rng, c.m, 9 * dim)).view(c.m, 9, dim)
    q, k, v = fused[:, :5], fused[:, 5:7], fused[:, 7:]
    pos = np.concatenate([np.arange(230, 300), np.arange(-1, 2), [63]]).astype(np.int32)
    one, two = c.cache(), c.cache()
    q_out = L.tern_kv_write(one, c.on_device(), k, v, rope=kr, q=q, q_rope=qr)
    turned = L.tern_rope(k, dev(pos), kr)
    L.tern_kv_write(two, c.on_device(), turned, v)
    assert torch.equal(one.k, two.k) and torch.equal(one.k_scale, two.k_scale) and torch.equal(one.v, two.v)
    want = L.tern_rope(q, dev(pos), qr)
    assert torch.equal(q_out, want)
    own = q.contiguous()
    assert L.tern_kv_write(two, c.on_device(), k, v, rope=kr, q=own, q_rope=qr, q_out=own) is own and torch.equal(own, want)

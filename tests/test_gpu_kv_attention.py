"""tern_kv_attention on the GPU against the oracle: rows and tiles, parts,
shared heads, windows, masks that leave a row empty, what lies in masked
places."""
import numpy as np
import pytest
import torch

from gpu_util import say
from kv_util import Case, check_attention, dev, half
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu


def run(c, q_heads, rng, scale=None, window=0, causal=True, max_len=None, q=None, note="", **kw):
    q = half(rng, c.m, q_heads, c.dim) if q is None else q
    scale = c.dim ** -0.5 if scale is None else scale
    cache, batch = c.cache(), c.on_device(max_len)
    out = torch.full((c.m, q_heads, c.dim), 55.0, dtype=torch.float16, device="cuda")
    got = L.tern_kv_attention(cache, batch, dev(q), scale=scale, window=window, causal=causal, out=out, **kw)
    check_attention(c, q, got, scale, window, causal, note)
    used = sum(c.rows)
    assert (got[used:] == 55).all(), "rows behind the last sequence changed"
    again = L.tern_kv_attention(cache, batch, dev(q), scale=scale, window=window, causal=causal)
    assert torch.equal(got[:used], again[:used]), "two runs differ"
    return got


ROWS = [
    # rows, lens, heads, query heads
    ([1], [1], 1, 1), ([1], [63], 2, 8), ([1], [64], 2, 2), ([1], [65], 3, 15), ([1, 1, 1], [700, 1, 129], 2, 8), ([2], [2], 1, 16),
    ([5, 2, 4], [300, 2, 68], 2, 6), ([3, 3], [2, 0], 1, 4), ([4], [2000], 1, 8), ([9], [200], 1, 7), ([1, 0, 2], [100, 3, 3], 2, 2),
    ([16], [500], 2, 2), ([17], [500], 1, 1), ([1], [5000], 1, 40), ([1], [130], 1, 64),
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,lens,heads,q_heads", ROWS)
def test_few_rows(rows, lens, heads, q_heads, dim):
    say("attention", rows, lens, heads, q_heads, dim)
    rng = np.random.default_rng(sum(rows) + sum(lens) + q_heads + dim)
    c = Case(rng, rows, lens, heads, dim, tail=3)
    run(c, q_heads, rng)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,lens,heads,q_heads", ROWS)
def test_few_rows_in_pieces(rows, lens, heads, q_heads, dim):
    """Cut into the line's pieces (by max_len), as long contexts are."""
    rng = np.random.default_rng(sum(rows) + sum(lens) + q_heads + dim)
    c = Case(rng, rows, lens, heads, dim, tail=3)
    run(c, q_heads, rng, max_len=10 ** 6)


@pytest.mark.parametrize("count,dim", [(3, 64), (60, 64), (130, 64), (3, 128), (60, 128), (130, 128), (3, 256), (40, 256), (70, 256)])
def test_units_shared_by_wavefronts(count, dim):
    """Eight, four and two wavefronts a unit; lengths of none to ten pages."""
    rng = np.random.default_rng(count + dim)
    lens = [0, 1, 64, 65, 640] + [int(n) for n in rng.integers(0, 641, count)]
    c = Case(rng, [2] * len(lens), lens, 8, dim)
    run(c, 16, rng)
    run(c, 16, rng, window=100)


TILES = [
    ([65], [65], 1, 1), ([70], [200], 1, 2), ([130], [130], 2, 4), ([33], [100], 1, 5), ([200, 3, 77], [333, 3, 400], 1, 3), ([129], [64], 1, 1),
    ([100, 100], [100, 0], 2, 2), ([90], [1500], 1, 4),
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,lens,heads,q_heads", TILES)
def test_tiles(rows, lens, heads, q_heads, dim):
    say("attention tiles", rows, lens, heads, q_heads, dim)
    rng = np.random.default_rng(sum(rows) + sum(lens) + q_heads + dim)
    c = Case(rng, rows, lens, heads, dim, tail=3)
    run(c, q_heads, rng)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 10 ** 6])
@pytest.mark.parametrize("rows,lens", [([1, 1], [500, 30]), ([5], [300]), ([100], [260])])
def test_windows(rows, lens, window):
    say("attention window", rows, lens, window)
    rng = np.random.default_rng(window + rows[0])
    run(Case(rng, rows, lens, 2, 64), 6, rng, window=window)


@pytest.mark.parametrize("rows,lens", [([1, 1], [500, 30]), ([5, 9, 2], [300, 1, 0]), ([100, 7], [260, 64]), ([200], [20])])
def test_not_causal(rows, lens):
    """An encoder's states: every row sees all of them, however many rows."""
    say("attention cross", rows, lens)
    rng = np.random.default_rng(rows[0])
    run(Case(rng, rows, lens, 2, 128), 4, rng, causal=False)


@pytest.mark.parametrize("rows", [1, 7, 100])
def test_scales_of_many_sizes(rows):
    """Pages' value scales over 2^16: the sums' units follow them."""
    for seed in range(3):
        rng = np.random.default_rng(seed)
        c = Case(rng, [rows], [900], 1, 64, spread=True)
        c.vs[rng.integers(0, len(c.vs), 2)] = 0
        c.ks[rng.integers(0, len(c.ks), 1)] = 0
        run(c, 2, rng, note=f"seed {seed}")


@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("spread", [0.0, 0.01, 30.0])
def test_flat_and_steep(rows, spread):
    """Scores all equal, and one token with nearly all the weight; scores that
    grow and fall along the context."""
    rng = np.random.default_rng(int(spread * 100))
    c = Case(rng, [rows], [1100], 1, 128)
    c.ks *= np.linspace(0.2, 3, len(c.ks))[:, None]
    c.ks = (c.ks.astype(np.float32).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32).astype(np.float64)
    q = (spread * rng.standard_normal((rows, 4, 128))).astype(np.float16)
    run(c, 4, rng, q=q)
    run(c, 4, rng, q=q, scale=0.0)


@pytest.mark.parametrize("rows", [1, 3, 90])
def test_small_weights_beside_a_large_one(rows):
    """Thousands of tokens with weights around FP16's smallest beside one
    with most: none is lost."""
    rng = np.random.default_rng(31)
    c = Case(rng, [rows], [3000], 1, 64)
    c.kc[:] = 0
    page, token = c.table[0, 3], 5
    c.kc[page, 0, token, 0] = 100
    c.ks[:] = 0.0625
    c.vc[:] = 100
    c.vc[page, 0, token] = -3
    q = np.zeros((rows, 1, 64), np.float16)
    q[:, :, 0] = 11.0 / (100 * 0.0625)  # weights e^-11 = 1.7e-5 of the large one
    run(c, 1, rng, q=q, scale=1.0)


def poison(c, seen):
    """NaN scales on every page that no row may see, garbage in the codes of
    every token behind the sequences' ends."""
    hidden = np.ones(len(c.ks), bool)
    hidden[[p for p in seen]] = False
    c.ks[hidden] = np.nan
    c.vs[hidden] = np.nan


@pytest.mark.parametrize("rows,lens,window", [([1, 1], [100, 64], 0), ([1], [500], 70), ([90], [500], 30), ([6], [64], 0), ([100], [100], 0)])
def test_what_lies_in_masked_places(rows, lens, window):
    """Spare pages, pages before the window and pages behind the end hold NaN
    scales: the results are those without them."""
    rng = np.random.default_rng(lens[0])
    c = Case(rng, rows, lens, 1, 64, extra=2)
    spare = sorted(set(range(len(c.ks))) - set(c.table[c.table >= 0].tolist()))
    c.table[:, -1] = spare[0]  # behind the end
    seen = set()
    for s, n in enumerate(lens):
        first = max(0, n - rows[s] - window + 1) if window else 0
        seen |= {int(c.table[s, t // 64]) for t in range(first, n)}
    poison(c, seen)
    run(c, 2, rng, window=window)


@pytest.mark.parametrize("rows", [8, 128])
def test_a_page_that_later_rows_alone_see(rows):
    """The last page is poisoned: rows before it are not touched by it, though
    they share its tile; the rows in it are NaN."""
    rng = np.random.default_rng(rows)
    c = Case(rng, [rows], [130], 1, 64)
    q = half(rng, rows, 2, 64)
    clean = L.tern_kv_attention(c.cache(), c.on_device(), dev(q))
    for bad in ("ks", "vs"):
        cache = c.cache()
        (cache.k_scale if bad == "ks" else cache.v_scale)[int(c.table[0, 2])] = np.nan
        got = L.tern_kv_attention(cache, c.on_device(), dev(q))
        assert torch.equal(got[:-2], clean[:-2]), bad
        assert torch.isnan(got[-2:]).all(), bad


def test_infinite_and_nan_queries_stay_in_their_rows():
    rng = np.random.default_rng(37)
    for rows in (4, 100):
        c = Case(rng, [rows], [200], 2, 64)
        q = half(rng, rows, 4, 64)
        clean = L.tern_kv_attention(c.cache(), c.on_device(), dev(q))
        q[2, 1, 5], q[3, 0, 0] = np.nan, np.inf
        got = L.tern_kv_attention(c.cache(), c.on_device(), dev(q))
        other = torch.ones(rows, 4, dtype=torch.bool)
        other[2, 1] = other[3, 0] = False
        assert torch.equal(got[other], clean[other]) and torch.isnan(got[2, 1]).all() and torch.isnan(got[3, 0]).all()


@pytest.mark.parametrize("rows,lens,q_heads", [([1, 1], [400, 300], 4), ([100], [400], 2)])
def test_pages_that_are_not_there(rows, lens, q_heads):
    rng = np.random.default_rng(41)
    c = Case(rng, rows, lens, 2, 64, holes=[(0, 1, -1), (0, 3, 10 ** 6)])
    run(c, q_heads, rng)
    c.table[:] = -1  # nothing at all
    run(c, q_heads, rng)


def test_query_strides():
    rng = np.random.default_rng(43)
    for rows in (1, 60):
        c = Case(rng, [rows] * 2, [300, 200], 2, 64)
        fused = dev(half(rng, c.m, 12 * 64)).view(c.m, 12, 64)
        q = fused[:, 1:7]
        cache, batch = c.cache(), c.on_device()
        assert torch.equal(L.tern_kv_attention(cache, batch, q), L.tern_kv_attention(cache, batch, q.contiguous()))


@pytest.mark.parametrize("rows", [1, 4, 80])
def test_parts_give_what_one_gives(rows):
    """max_len chooses the number of parts, not the result."""
    rng = np.random.default_rng(47)
    c = Case(rng, [rows], [3000], 1, 128)
    q = half(rng, rows, 2, 128)
    for max_len in (0, 64, 600, None, 10 ** 6):
        run(c, 2, rng, q=q, max_len=max_len, note=f"max_len {max_len}")


@pytest.mark.parametrize("rows,most", [([1, 2], 500), ([30, 50], 2000)])
def test_more_rows_announced_than_there_are(rows, most):
    rng = np.random.default_rng(44)
    c = Case(rng, rows, [700, 900], 2, 64, ragged=True, tail=1)
    c.max_rows = most
    run(c, 4, rng)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,lens,q_heads", [([17], [500], 1), ([5, 2, 4], [300, 2, 68], 4), ([8, 8], [700, 7], 4), ([1, 1], [900, 65], 32)])
def test_two_blocks_of_rows(rows, lens, q_heads, dim):
    """17 to 32 rows of a cache head, with pages enough (by max_len) for the
    kernel for few rows."""
    rng = np.random.default_rng(46)
    c = Case(rng, rows, lens, 1, dim)
    for max_len in (None, 10 ** 6):
        run(c, q_heads, rng, max_len=max_len, note=f"max_len {max_len}")


@pytest.mark.parametrize("window", [0, 40])
def test_two_blocks_of_rows_of_many_sequences(window):
    rng = np.random.default_rng(49)
    lens = [int(n) for n in rng.integers(5, 193, 180)]
    run(Case(rng, [5] * 180, lens, 8, 64), 32, rng, window=window)


@pytest.mark.parametrize("dim,rows", [(64, 1), (128, 3)])
def test_many_short_sequences(dim, rows):
    """More units than 64 for every page: a wavefront each; cut by a max_len
    that leaves too few."""
    rng = np.random.default_rng(48)
    lens = [int(n) for n in rng.integers(0, 513, 77)] + [512, 1, 64]
    c = Case(rng, [rows] * len(lens), [n + rows for n in lens], 8, dim)
    q = half(rng, c.m, 32, dim)
    for max_len in (None, 8192):
        run(c, 32, rng, q=q, max_len=max_len, note=f"max_len {max_len}")


def test_long_context():
    """A table of 2^15 pages over few pages of memory: positions past 10^6."""
    rng = np.random.default_rng(53)
    c = Case(rng, [2], [200], 1, 64)
    tokens = 1 << 21
    table = np.resize(c.table[0, :4], tokens // 64).astype(np.int32)[None]
    batch = L.KvBatch(dev(np.array([tokens], np.int32)), dev(table), 2)
    q = half(rng, 2, 2, 64)
    got = L.tern_kv_attention(c.cache(), batch, dev(q)).float().cpu().numpy()
    # every page is seen 2^21 / 256 times: the softmax over the four, the second row whole
    p = c.table[0, :4]
    k, v = ((x[p, 0] * f[p, 0][:, None, None]).reshape(256, 64) for x, f in ((c.kc, c.ks), (c.vc, c.vs)))
    z = k @ q[1].astype(np.float64).T / 8
    w = np.exp(z - z.max(axis=0))
    want = (w / w.sum(axis=0)).T @ v
    size = (w / w.sum(axis=0)).T @ np.abs(v)
    # weights' and outputs' roundings, scores' FP32, and sums of 2^21 weights in
    # chains of at most 2^21 / 4 / 4 pages' partial sums
    assert (np.abs(got[1] - want) <= 2.0 ** -11 * np.abs(want) + size * (2.0 ** -11 + 2.0 ** -23 * (2.0 ** 14 + 400)) + 1e-6).all()


def test_cache_past_32_bits():
    """A cache of more than 2^32 bytes: the last page is written, read and
    attended to."""
    rng = np.random.default_rng(59)
    heads, dim = 8, 128
    pages = (1 << 32) // (heads * 64 * dim) + 3
    k, v = (torch.full((pages, heads, 64, dim), 128, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, heads), device="cuda") for _ in range(2))
    cache = L.KvCache(k, v, ks, vs)
    batch = L.KvBatch(dev(np.array([3], np.int32)), dev(np.array([[pages - 1]], np.int32)), 3)
    kk, vv = half(rng, 3, heads, dim), half(rng, 3, heads, dim)
    L.tern_kv_write(cache, batch, dev(kk), dev(vv))
    back = L.tern_kv_read(cache, batch)
    assert (np.abs(back[1].cpu().numpy() - vv) <= np.abs(vv).max() / 120).all()
    assert int((ks != 0).sum()) == heads and (ks[pages - 1] > 0).all()
    y = L.tern_kv_attention(cache, batch, dev(half(rng, 3, heads, dim)))
    assert torch.equal(y[0], back[1][0])  # the first row sees one token: its value

"""Attention in the forms that differ by head size and kernel: windows, rows
that are not causal, what lies in masked places, and pages that are not there,
for every head size on few rows, on tiles of 64 and of 128 rows; batches that
mix a prompt's chunk with single tokens."""
import numpy as np
import pytest
import torch

import test_gpu_kv_attention as A
from gpu_util import say
from kv_util import Case, dev, half
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu

DIMS = [64, 128, 256]


@pytest.fixture(params=["few rows", 64, 128])
def kernel(request):
    """The kernel for few rows, or the tiles' rows."""
    if request.param != "few rows":
        L.tern_kv_tile_rows(request.param)
    yield request.param
    L.tern_kv_tile_rows(0)


def many(kernel, few, rows):
    return few if kernel == "few rows" else rows


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("window", [1, 63, 64, 65, 200, 10 ** 6])
def test_windows(kernel, window, dim):
    say("window", kernel, window, dim)
    rng = np.random.default_rng(window + dim)
    for rows, lens in many(kernel, [([1, 1], [500, 30]), ([5], [300])], [([100], [260]), ([70, 40], [900, 41])]):
        A.run(Case(rng, rows, lens, 2, dim), 6, rng, window=window, note=f"{rows}")


@pytest.mark.parametrize("dim", DIMS)
def test_not_causal(kernel, dim):
    say("not causal", kernel, dim)
    rng = np.random.default_rng(dim)
    for rows, lens in many(kernel, [([1, 1], [500, 30]), ([5, 3, 2], [300, 1, 0])], [([100, 7], [260, 64]), ([200], [20]), ([70, 90], [1000, 0])]):
        A.run(Case(rng, rows, lens, 2, dim), 4, rng, causal=False, note=f"{rows}")


@pytest.mark.parametrize("dim", DIMS)
def test_what_lies_in_masked_places(kernel, dim):
    """NaN scales of spare pages, of pages before the window and behind the end."""
    say("masked", kernel, dim)
    for rows, lens, window in many(kernel, [([1, 1], [100, 64], 0), ([1], [500], 70), ([6], [64], 0)], [([90], [500], 30), ([100], [100], 0), ([70], [300], 65)]):
        rng = np.random.default_rng(lens[0] + dim)
        c = Case(rng, rows, lens, 1, dim, extra=2)
        c.table[:, -1] = sorted(set(range(len(c.ks))) - set(c.table[c.table >= 0].tolist()))[0]
        seen = set()
        for s, n in enumerate(lens):
            first = max(0, n - rows[s] - window + 1) if window else 0
            seen |= {int(c.table[s, t // 64]) for t in range(first, n)}
        A.poison(c, seen)
        A.run(c, 2, rng, window=window, note=f"{rows}")


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("bad", ["ks", "vs"])
def test_a_page_that_later_rows_alone_see(kernel, bad, dim):
    rng = np.random.default_rng(dim)
    c = Case(rng, [many(kernel, 8, 128)], [130], 1, dim)
    q = half(rng, c.m, 2, dim)
    clean = L.tern_kv_attention(c.cache(), c.on_device(), dev(q))
    cache = c.cache()
    (cache.k_scale if bad == "ks" else cache.v_scale)[int(c.table[0, 2])] = np.nan
    got = L.tern_kv_attention(cache, c.on_device(), dev(q))
    assert torch.equal(got[:-2], clean[:-2]) and torch.isnan(got[-2:]).all()


@pytest.mark.parametrize("dim", DIMS)
def test_pages_before_a_window_do_not_matter(kernel, dim):
    """Rows of a tile whose windows begin on different pages: a NaN page that
    the first rows see leaves the others as they are."""
    rng = np.random.default_rng(dim)
    rows, window = many(kernel, 16, 128), 40
    c = Case(rng, [rows], [rows + 200], 1, dim)
    q = half(rng, rows, 1, dim)
    first = 200 - window + 1  # the first row's first token
    clean = L.tern_kv_attention(c.cache(), c.on_device(), dev(q), window=window)
    for bad in ("k_scale", "v_scale"):
        cache = c.cache()
        getattr(cache, bad)[int(c.table[0, first // 64])] = np.nan
        got = L.tern_kv_attention(cache, c.on_device(), dev(q), window=window)
        hit = torch.tensor([(200 + r - window + 1) // 64 <= first // 64 for r in range(rows)])
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit]), bad


@pytest.mark.parametrize("dim", DIMS)
def test_infinite_and_nan_queries_stay_in_their_rows(kernel, dim):
    rng = np.random.default_rng(dim)
    rows = many(kernel, 4, 100)
    c = Case(rng, [rows], [200], 2, dim)
    q = half(rng, rows, 4, dim)
    clean = L.tern_kv_attention(c.cache(), c.on_device(), dev(q))
    q[2, 1, 5], q[3, 0, 0] = np.nan, np.inf
    got = L.tern_kv_attention(c.cache(), c.on_device(), dev(q))
    other = torch.ones(rows, 4, dtype=torch.bool)
    other[2, 1] = other[3, 0] = False
    assert torch.equal(got[other], clean[other]) and torch.isnan(got[2, 1]).all() and torch.isnan(got[3, 0]).all()


@pytest.mark.parametrize("dim", DIMS)
def test_pages_that_are_not_there(kernel, dim):
    rng = np.random.default_rng(dim)
    rows, lens = many(kernel, ([1, 1], [400, 300]), ([100], [400]))
    c = Case(rng, rows, lens, 2, dim, holes=[(0, 1, -1), (0, 3, 10 ** 6)])
    A.run(c, 4, rng)
    A.run(c, 4, rng, window=70)
    A.run(c, 4, rng, causal=False)
    c.table[:] = -1  # nothing at all
    A.run(c, 4, rng)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("rows,lens,heads,q_heads", [
    ([130, 1, 1, 1], [190, 3000, 64, 1], 2, 8), ([1, 1, 70, 1, 0, 9], [700, 65, 70, 0, 5, 900], 1, 4), ([1, 40, 1], [20000, 300, 129], 2, 4)])
def test_chunks_of_prompts_beside_single_tokens(kernel, rows, lens, heads, q_heads, dim):
    """One call, by the rule and on either tile; the longest sequence chooses
    the kernel."""
    say("mixed", kernel, rows, lens, dim)
    rng = np.random.default_rng(sum(rows) + dim)
    A.run(Case(rng, rows, lens, heads, dim, tail=2), q_heads, rng)


@pytest.mark.parametrize("dim", DIMS)
def test_a_mixed_batch_gives_what_calls_apart_give(dim):
    """Each sequence in a call of its own, on the kernel that it takes there: off
    by both calls' bounds at most."""
    rng = np.random.default_rng(dim)
    rows, lens = [150, 1, 1], [400, 2500, 77]
    c = Case(rng, rows, lens, 2, dim)
    q = half(rng, c.m, 8, dim)
    A.run(c, 8, rng, q=q)
    cache, at = c.cache(), 0
    for s, n in enumerate(rows):
        one = Case.__new__(Case)
        one.__dict__.update(c.__dict__, rows=[n], lens=[lens[s]], table=c.table[s:s + 1], max_rows=n, start=None, m=n)
        got = L.tern_kv_attention(cache, one.on_device(), dev(q[at:at + n]))
        A.check_attention(one, q[at:at + n], got, dim ** -0.5, note=f"sequence {s}")
        at += n

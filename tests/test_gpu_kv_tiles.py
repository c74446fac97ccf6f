"""Attention on tiles of 64 and of 128 rows: every check that test_gpu_kv_attention
makes of calls with many rows, with either kernel, and prompts by the rule."""
import numpy as np
import pytest

import test_gpu_kv_attention as A
from kv_util import Case
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[64, 128])
def tile(request):
    L.tern_kv_tile_rows(request.param)
    yield request.param
    L.tern_kv_tile_rows(0)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows,lens,heads,q_heads", A.TILES + [([33], [33], 1, 1), ([64, 1, 128], [64, 900, 500], 2, 2), ([9], [5000], 1, 7)])
def test_tiles(tile, rows, lens, heads, q_heads, dim):
    A.test_tiles(rows, lens, heads, q_heads, dim)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 10 ** 6])
@pytest.mark.parametrize("rows,lens", [([100], [260]), ([70, 40], [900, 41])])
def test_windows(tile, rows, lens, window):
    A.test_windows(rows, lens, window)


@pytest.mark.parametrize("rows,lens", [([100, 7], [260, 64]), ([200], [20])])
def test_not_causal(tile, rows, lens):
    A.test_not_causal(rows, lens)


def test_scales(tile):
    A.test_scales_of_many_sizes(100)


@pytest.mark.parametrize("spread", [0.0, 0.01, 30.0])
def test_flat_and_steep(tile, spread):
    A.test_flat_and_steep(90, spread)


def test_small_weights_beside_a_large_one(tile):
    A.test_small_weights_beside_a_large_one(90)


@pytest.mark.parametrize("rows,lens,window", [([90], [500], 30), ([100], [100], 0)])
def test_what_lies_in_masked_places(tile, rows, lens, window):
    A.test_what_lies_in_masked_places(rows, lens, window)


def test_a_page_that_later_rows_alone_see(tile):
    A.test_a_page_that_later_rows_alone_see(128)


def test_infinite_and_nan_queries_stay_in_their_rows(tile):
    A.test_infinite_and_nan_queries_stay_in_their_rows()


def test_pages_that_are_not_there(tile):
    A.test_pages_that_are_not_there([100], [400], 2)


@pytest.mark.parametrize("rows,most", [([30, 50], 2000)])
def test_more_rows_announced_than_there_are(tile, rows, most):
    A.test_more_rows_announced_than_there_are(rows, most)


def test_parts(tile):
    A.test_parts_give_what_one_gives(80)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_more_than_32_parts(tile, dim):
    """One cache head's long contexts, of which a tile's last rows alone see the
    last page."""
    rng = np.random.default_rng(dim)
    A.run(Case(rng, [40, 70], [4700, 3000], 1, dim), 1, rng)


@pytest.mark.parametrize("rows,lens,heads,q_heads", [([300, 200], [300, 700], 2, 8), ([400] * 4, [450] * 4, 8, 16)])
def test_by_the_rule(rows, lens, heads, q_heads):
    rng = np.random.default_rng(len(rows))
    A.run(Case(rng, rows, lens, heads, 128), q_heads, rng)

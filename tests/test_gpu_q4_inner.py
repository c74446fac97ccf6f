"""tern_q4_experts on the GPU: the inner values silu(g) * u keep FP32's range
and some 17 bits or more on each of the routes, however small or large they
are."""
import numpy as np
import pytest

from gpu_util import say, to_dev
from oracle import q4_oracle as Q
from q4_util import check, half, kind_of, upload, weights
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu

# m, topk, experts: slot by slot, tiles of 16, 32 and 64 rows
ROUTES = [(1, 8, 16), (4, 4, 8), (30, 2, 20), (60, 2, 7), (420, 2, 2)]


def setting(rng, m, topk, count, group, zero, hidden=256, inner=256, width=40):
    up, down = weights(rng, (count,), 2 * inner, hidden, group, zero), weights(rng, (count,), width, inner, group, zero)
    ids = np.stack([rng.permutation(max(count, topk))[:topk] for _ in range(m)]).astype(np.int32) % count
    return up, down, ids, rng.uniform(0.01, 1, (m, topk)).astype(np.float32), rng.standard_normal((m, hidden))


def run(up, down, x, ids, g, out):
    return L.tern_q4_experts(upload(up), upload(down), half(x), to_dev(ids), to_dev(g), kind_of(out))


@pytest.mark.parametrize("group,zero", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("m,topk,count", ROUTES)
@pytest.mark.parametrize("size", [1e-3, 0.1, 1.0, 1e5])
def test_inner_values_of_any_size(size, m, topk, count, group, zero):
    """Gate and up projections near `size`: inner values near 1e-6 (below
    FP16's normal range) up to 1e10 (far above it)."""
    say("inner", size, m, topk, count, group, zero)
    rng = np.random.default_rng(m + group)
    up, down, ids, g, x = setting(rng, m, topk, count, group, zero)
    # a projection of 256 unit normals at scales near 0.01 is near 1: x and the scales share the rest
    by = min(size, 100.0)
    x = (x * by).astype(np.float16)
    up = (up[0], (up[1].astype(np.float64) * (size / by)).astype(np.float16), up[2])
    y, err = Q.experts(up, down, group, x, ids, g, parts=2 if m * topk <= 32 else 1)
    check(run(up, down, x, ids, g, "f32"), y, err, "f32", "inner f32")
    # scales that bring an FP16 output to ordinary size
    s = np.clip(down[1].astype(np.float64) / np.abs(y).mean(), 2.0 ** -14, 6e4).astype(np.float16)
    down = (down[0], s, down[2])
    y, err = Q.experts(up, down, group, x, ids, g, parts=2 if m * topk <= 32 else 1)
    if np.abs(y).max() < 6e4:
        check(run(up, down, x, ids, g, "f16"), y, err, "f16", "inner f16")


@pytest.mark.parametrize("m,topk,count", ROUTES)
def test_large_inner_values_meet_zero_weights(m, topk, count):
    """Inner values beyond 65504 beside down weights of zero: exact sums."""
    up = (np.full((count, 64, 64), 15, np.uint8), np.full((count, 64, 2), 4.0, np.float16), None)  # weights 28
    d = np.full((count, 3, 32), 9, np.uint8)  # weights 1, every other one 0
    d[:, :, 1::2] = 8
    down = (d, np.ones((count, 3, 1), np.float16), None)
    x = np.ones((m, 64), np.float16)
    ids = (np.arange(m * topk, dtype=np.int32) % count).reshape(m, topk)
    got = run(up, down, x, ids, np.ones((m, topk), np.float32), "f32").cpu().numpy()
    # gate = up = 64 * 28, silu(1792) = 1792; 16 weights of 1 a slot; every partial sum is below 2^24 units of 2^16
    assert (got == topk * 16 * 1792.0 ** 2).all()


@pytest.mark.parametrize("m,topk,count", ROUTES)
def test_inner_values_past_range_are_infinite(m, topk, count):
    """Beyond 2^71 an inner value is infinite: with weights of one sign an
    infinite output, no NaN."""
    import torch
    up = (np.full((count, 64, 128), 0, np.uint8), np.full((count, 64, 2), 60000.0, np.float16), np.full((count, 64, 2), 255, np.uint8))
    down = (np.full((count, 3, 32), 9, np.uint8), np.ones((count, 3, 1), np.float16), None)
    x = np.full((m, 128), -60000.0, np.float16)  # gate and up 1.2e14 each: inner 1.4e28
    ids = (np.arange(m * topk, dtype=np.int32) % count).reshape(m, topk)
    assert torch.isposinf(run(up, down, x, ids, np.ones((m, topk), np.float32), "f32")).all()


@pytest.mark.parametrize("m,topk,count", ROUTES)
@pytest.mark.parametrize("gate", [1e-30, 1e30])
def test_weights_of_any_size(gate, m, topk, count):
    """A slot's weight far from 1: outputs keep FP32's range."""
    rng = np.random.default_rng(m)
    up, down, ids, g, x = setting(rng, m, topk, count, 64, True)
    x, g = x.astype(np.float16), (g * gate).astype(np.float32)
    y, err = Q.experts(up, down, 64, x, ids, g, parts=2 if m * topk <= 32 else 1)
    check(run(up, down, x, ids, g, "f32"), y, err, "f32", f"weights near {gate}")

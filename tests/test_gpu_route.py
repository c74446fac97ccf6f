"""tern_route on the GPU against the oracle: the same experts in the same
order, weights within their rounding to FP32."""
import numpy as np
import pytest

from gpu_util import say, to_dev
from oracle import q4_oracle as Q
from q4_util import replay_checks
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu

SCORE = {"softmax": L.TERN_SCORE_SOFTMAX, "sigmoid": L.TERN_SCORE_SIGMOID}


def run(l, topk, score="softmax", bias=None, groups=1, best=1, keep=1, renorm=True, scale=1.0):
    """Routes on the GPU and compares; returns the ids."""
    ids, w = L.tern_route(to_dev(l), topk, SCORE[score], None if bias is None else to_dev(bias), groups, best, keep, renorm, scale)
    want, g = Q.route(l, topk, score, bias, groups, best, keep, renorm, scale)
    ids, w = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    assert np.array_equal(ids, want), f"ids differ in rows {np.argwhere((ids != want).any(1))[:5].ravel()}"
    # FP64 up to its rounding, then half a step of FP32
    assert (np.abs(w - g) <= np.abs(g) * 2.0 ** -24 * 1.001 + 2.0 ** -149).all()
    return ids


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,experts,topk,groups,best,keep", [
    (1, 1, 1, 1, 1, 1), (1, 8, 2, 1, 1, 1), (5, 60, 4, 1, 2, 1), (37, 64, 8, 8, 2, 3), (130, 256, 8, 8, 2, 4),
    (9, 160, 6, 8, 1, 3), (3, 257, 64, 1, 1, 1), (4, 512, 10, 16, 2, 5), (2, 1000, 8, 4, 2, 2), (3, 1024, 16, 64, 1, 9),
    (6, 128, 1, 64, 2, 1), (7, 96, 12, 3, 2, 1)])
def test_route_matches_oracle(m, experts, topk, groups, best, keep, score, dtype):
    say("route", m, experts, topk, groups, best, keep, score, dtype.__name__)
    rng = np.random.default_rng(m + experts)
    for bias in (None, (0.1 * rng.standard_normal(experts)).astype(np.float32)):
        for renorm, scale in ((True, 2.5), (False, 1.0)):
            l = (2 * rng.standard_normal((m, experts))).astype(dtype)
            run(l, topk, score, bias, groups, best, keep, renorm, scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_and_odd_logits(score):
    rng = np.random.default_rng(1)
    for dtype in (np.float16, np.float32):
        l = rng.standard_normal((40, 48)).astype(dtype)
        l[rng.random(l.shape) < 0.3] = -np.inf
        l[rng.random(l.shape) < 0.05] = np.nan
        l[3] = -np.inf
        l[4] = np.nan
        l[5, :2] = np.inf
        l[6, 1:] = -np.inf
        bias = rng.standard_normal(48).astype(np.float32)
        bias[[1, 2, 3]] = np.nan, -np.inf, np.inf
        for b in (None, bias):
            for groups, best, keep in ((1, 1, 1), (6, 2, 2), (6, 1, 5)):
                ids = run(l, 8, score, b, groups, best, keep)
                assert (ids[3] == -1).all() and (ids[4] == -1).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest(score):
    rng = np.random.default_rng(2)
    l = rng.integers(-2, 3, (60, 128)).astype(np.float16)
    l[l == 0] *= rng.choice([-1, 1], (l == 0).sum()).astype(np.float16)  # -0 ties with 0
    flat = np.zeros(128, np.float32)
    for b in (None, flat):
        for groups, best, keep in ((1, 1, 1), (8, 2, 3)):
            run(l, 16, score, b, groups, best, keep)
            run(l.astype(np.float32), 16, score, b, groups, best, keep)


def test_route_keys_that_fp32_cannot_tell_apart():
    """Sigmoids near 1 and softmax scores far below the largest."""
    l = np.linspace(17, 20, 64).astype(np.float32)[None].repeat(3, 0)
    l[1] = l[1][::-1]
    run(l, 8, "sigmoid", np.zeros(64, np.float32), 8, 2, 3)
    l = np.linspace(-150, -100, 64).astype(np.float32)[None].repeat(2, 0)
    l[:, 5] = 0
    bias = np.zeros(64, np.float32)
    bias[5] = -9
    run(l, 4, "softmax", bias)
    run(np.full((2, 32), -120, np.float32) - np.arange(32, dtype=np.float32), 4, "sigmoid", None, 4, 2, 2)


@pytest.mark.parametrize("experts,groups,topk", [(64, 4, 6), (128, 2, 8), (256, 8, 8), (200, 5, 12)])
def test_route_near_ties(experts, groups, topk):
    """Keys a few FP32 steps apart, in any order, beside clear ones; biases
    that cancel the scores' differences; biases far out."""
    rng = np.random.default_rng(experts)
    for score in ("softmax", "sigmoid"):
        l = rng.standard_normal((40, experts)).astype(np.float32)
        l[::2] = np.float32(1.25) + rng.integers(-6, 7, l[::2].shape).astype(np.float32) * np.float32(2.0 ** -23)
        run(l, topk, score)
        run(l, topk, score, np.zeros(experts, np.float32), groups, 2, max(1, groups // 2))
        run(l, topk, score, (rng.integers(-3, 4, experts) * 2.0 ** -24).astype(np.float32), groups, 1, groups)
        run(l, topk, score, (10 * rng.standard_normal(experts)).astype(np.float32), groups, 2, groups)
        run(l, topk, score, None, groups, 2, 1 if topk <= experts // groups else 2, renorm=False)
        run((1e-30 * l).astype(np.float32), topk, score)


def test_route_of_more_tokens_than_a_launch():
    import torch
    gen = torch.Generator(device="cuda").manual_seed(5)
    l = torch.randn(((1 << 24) + 777, 2), device="cuda", generator=gen).half()
    ids, w = L.tern_route(l, 1, scale=0.5)
    assert torch.equal(ids[:, 0], (l[:, 1] > l[:, 0]).int()) and (w == 0.5).all()


def test_route_captured():
    import torch
    l = torch.randn((33, 64), device="cuda")
    ids = torch.empty((33, 6), dtype=torch.int32, device="cuda")
    w = torch.empty((33, 6), device="cuda")
    replay_checks(lambda s: L.tern_route(l, 6, ids=ids, weights=w, stream=s), lambda r: l.normal_(), [ids, w])


def test_route_writes_its_outputs_alone():
    import torch
    l = torch.randn((5, 100), device="cuda")
    ids = torch.full((7, 3), -9, dtype=torch.int32, device="cuda")
    w = torch.full((7, 3), -9.0, device="cuda")
    L.tern_route(l, 3, ids=ids[1:-1], weights=w[1:-1])
    for t in (ids, w):
        assert (t[0] == -9).all() and (t[-1] == -9).all() and (t[1:-1] != -9).all()
    got, _ = L.tern_route(torch.empty((0, 8), device="cuda"), 2)
    assert got.shape == (0, 2)


def test_route_refusals_of_tensors():
    import torch
    l = torch.randn((4, 8), device="cuda")
    for bad in (l.cpu(), l.double(), l.t(), l[0]):
        with pytest.raises(ValueError):
            L.tern_route(bad, 2)
    with pytest.raises(ValueError):
        L.tern_route(l, 2, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        L.tern_route(l, 2, ids=torch.zeros((4, 3), dtype=torch.int32, device="cuda"))
    with pytest.raises(L.TernError):
        L.tern_route(l, 9)

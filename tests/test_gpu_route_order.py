"""tern_route without a bias, groups judged by their two best: the groups go
by their scores' sums, the experts by their logits, also where the scores
cannot be told apart."""
import numpy as np
import pytest

from gpu_util import say
from test_gpu_route import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,topk", [(8, 2, 3), (64, 8, 8), (64, 2, 12), (128, 4, 9), (256, 8, 8), (160, 8, 6), (512, 16, 10)])
def test_experts_go_by_their_logits(experts, groups, topk, score, dtype):
    """Sigmoids of 36 and more are 1 but for FP64's last bits, softmax scores
    800 below the largest are 0."""
    say("order", experts, groups, topk, score, dtype.__name__)
    rng = np.random.default_rng(experts + topk)
    m = 33
    far = np.stack([rng.permutation(experts) for _ in range(m)])
    l = (36 + far * (24 / experts) if score == "sigmoid" else -2.0 * far - 800).astype(dtype)
    if score == "softmax":
        l[:, 0] = 0
    ids = run(l, topk, score, None, groups, 2, groups)
    assert np.array_equal(ids, np.argsort(-l.astype(np.float64), axis=1, kind="stable")[:, :topk])
    for keep in range(max(1, -(-topk // (experts // groups))), groups):
        run(l, topk, score, None, groups, 2, keep, renorm=keep % 2 == 0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,topk", [(64, 8, 8), (128, 4, 9), (256, 8, 8), (160, 8, 6)])
def test_groups_go_by_their_sums(experts, groups, topk, score):
    """Ordinary, close and masked logits, every number of groups kept."""
    rng = np.random.default_rng(experts)
    for dtype in (np.float16, np.float32):
        for scale in (1e-3, 1.0, 12.0):
            l = (scale * rng.standard_normal((40, experts))).astype(dtype)
            l[rng.random(l.shape) < 0.2] = -np.inf
            l[3] = -np.inf
            l[4] = l[4, 0] if np.isfinite(l[4, 0]) else 1
            for keep in range(max(1, -(-topk // (experts // groups))), groups + 1):
                run(l, topk, score, None, groups, 2, keep, renorm=keep % 2 == 0)


def test_the_larger_of_two_saturated_scores_comes_first():
    l = np.zeros((1, 8), np.float32)
    l[0, 1], l[0, 5] = 40, 50
    assert run(l, 2, "sigmoid", None, 2, 2, 2).tolist() == [[5, 1]]
    l = np.full((1, 8), -1000, np.float32)
    l[0, 2], l[0, 7] = 0, -900
    assert run(l, 2, "softmax", None, 2, 2, 2).tolist() == [[2, 7]]


def test_settings_past_32_bits_are_refused():
    import torch
    from ternary_weight_only_tern_amd import lib as L
    l = torch.randn((4, 8), device="cuda")
    far = 1 << 32
    for kw in (dict(topk=far + 2), dict(groups=far + 1), dict(groups=2, keep_groups=far + 1), dict(group_best=far + 1)):
        with pytest.raises(ValueError):
            L.tern_route(l, **{**dict(topk=2), **kw})

"""The 4-bit layers' oracle against hand-worked values and brute force."""
import itertools
import math

import numpy as np
import pytest

from oracle import q4_oracle as Q


def test_pack_word_by_hand():
    # offsets 0..7 in bits 0, 16, 4, 20, 8, 24, 12, 28
    assert Q.pack(np.arange(8, dtype=np.uint8)).view("<u4").tolist() == [0x75316420]
    assert Q.pack(np.array([15, 0, 0, 0, 0, 0, 0, 1], np.uint8)).tolist() == [0x0F, 0, 0, 0x10]


def test_gemm_is_the_dense_product():
    rng = np.random.default_rng(0)
    q = rng.integers(0, 16, (3, 64), dtype=np.uint8)
    s = rng.uniform(0.1, 1, (3, 2)).astype(np.float16)
    z = rng.integers(0, 256, (3, 2), dtype=np.uint8)
    x = rng.standard_normal((2, 64)).astype(np.float16)
    y, b, _ = Q.gemm(q, s, z, 32, x)
    for i, n in itertools.product(range(2), range(3)):
        terms = [float(s[n, k // 32]) * (int(q[n, k]) - int(z[n, k // 32])) * float(x[i, k]) for k in range(64)]
        assert math.isclose(y[i, n], math.fsum(terms), rel_tol=1e-12, abs_tol=1e-12)
        assert math.isclose(b[i, n], math.fsum(map(abs, terms)), rel_tol=1e-12)
    assert np.allclose(Q.gemm(q, s, None, 32, x)[0], Q.gemm(q, s, np.full((3, 2), 8, np.uint8), 32, x)[0])


@pytest.mark.parametrize("score,bias,groups,best,keep", [("softmax", False, 1, 1, 1), ("sigmoid", True, 3, 2, 2),
                                                         ("softmax", True, 2, 1, 1), ("sigmoid", False, 2, 2, 1)])
def test_route_takes_the_best_subset(score, bias, groups, best, keep):
    """Of every way to keep groups and choose experts, the one chosen has the
    largest sums."""
    rng = np.random.default_rng(3)
    experts, topk, size = 6, 2, 6 // groups
    l = rng.standard_normal((5, experts)).astype(np.float32)
    b = rng.standard_normal(experts).astype(np.float32) * 0.2 if bias else None
    ids, w = Q.route(l, topk, score, b, groups, best, keep, True, 2.5)
    for t in range(5):
        v = l[t].astype(np.float64)
        s = 1 / (1 + np.exp(-v)) if score == "sigmoid" else np.exp(v) / np.exp(v).sum()
        key = s + (0 if b is None else b.astype(np.float64))
        judge = lambda g: sum(sorted(key[g * size:(g + 1) * size])[-best:])
        kept = max(itertools.combinations(range(groups), keep), key=lambda c: sum(map(judge, c)))
        of = [e for e in range(experts) if e // size in kept]
        pair = max(itertools.combinations(of, topk), key=lambda c: sum(key[list(c)]))
        assert sorted(ids[t]) == sorted(pair)
        assert key[ids[t, 0]] >= key[ids[t, 1]]
        assert np.allclose(w[t], 2.5 * s[ids[t]] / s[ids[t]].sum())


def test_route_masks_ties_and_odd_values():
    inf, nan = np.inf, np.nan
    l = np.array([[1, 1, 1, 1], [-inf, nan, 2, -inf], [-inf] * 4, [inf, 0, inf, 5]], np.float32)
    ids, w = Q.route(l, 2)
    assert ids.tolist() == [[0, 1], [2, -1], [-1, -1], [0, 2]]
    assert w.tolist() == [[0.5, 0.5], [1, 0], [0, 0], [0.5, 0.5]]
    ids, w = Q.route(l[:1], 3, "sigmoid", np.array([nan, -inf, 0, inf], np.float32), renorm=False)
    assert ids.tolist() == [[3, 2, -1]]


def test_experts_by_hand():
    """One weight wide: y = gate * wd * silu(wg x) * (wu x)."""
    k = 32
    q = np.full((2, 2 * k, k), 8, np.uint8)
    s = np.ones((2, 2 * k, 1), np.float16)
    q[1, 0, 0], q[1, k, 0] = 10, 11  # expert 1: gate 2 x0, up 3 x0 in inner channel 0
    qd = np.full((2, 1, k), 8, np.uint8)
    qd[1, 0, 0] = 7  # down: minus channel 0
    x = np.zeros((1, k), np.float16)
    x[0, 0] = 0.5
    y, err = Q.experts((q, s, None), (qd, np.ones((2, 1, 1), np.float16), None), 32, x, np.array([[1, -1, 1, 2]]),
                       np.array([[0.25, 9, 0.5, 9]], np.float32))
    want = -0.75 * (1 / (1 + math.exp(-1))) * 1.5
    assert math.isclose(y[0, 0], want, rel_tol=1e-12)
    assert 0 < err[0, 0] < 2e-3


def test_route_without_a_bias_goes_by_the_logits():
    """Scores that FP64 cannot tell apart: the larger logit is chosen first,
    and groups judged by two such experts tie, so that the lower one stays."""
    l = np.zeros((1, 8), np.float32)
    l[0, 1], l[0, 5] = 40, 50
    assert Q.route(l, 2, "sigmoid", None, 2, 2, 2)[0].tolist() == [[5, 1]]
    l[0, 0:2], l[0, 4:6] = (40, 41), (50, 51)
    assert Q.route(l, 1, "sigmoid", None, 2, 2, 1)[0].tolist() == [[1]]
    l = np.full((1, 8), -1000, np.float32)
    l[0, 2], l[0, 7] = 0, -900
    assert Q.route(l, 2, "softmax", None, 2, 2, 2)[0].tolist() == [[2, 7]]

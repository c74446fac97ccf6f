"""Pins of oracle/kv_oracle.py: closed forms, brute force, invariants."""
import numpy as np
import pytest

from oracle import kv_oracle as K


@pytest.mark.parametrize("keys", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_places_are_a_permutation(dim, keys):
    at = K.place(dim, keys)
    assert np.array_equal(np.sort(at, axis=None), np.arange(64 * dim))
    codes = np.random.default_rng(0).integers(-127, 128, (2, 3, 64, dim))
    assert np.array_equal(K.unpack(K.pack(codes, keys), dim, keys), codes)


def test_places_by_hand():
    k, v = K.place(128, True), K.place(128, False)
    assert [k[0, 0], k[0, 15], k[1, 0], k[4, 0], k[16, 0], k[0, 16], k[0, 64], k[63, 127]] == [0, 15, 16, 1024, 64, 256, 4096, 8191]
    assert [v[0, 0], v[15, 0], v[0, 1], v[16, 0], v[0, 16], v[63, 127]] == [0, 15, 16, 256, 1024, 8191]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_keeps_lengths_and_differences(interleaved):
    rng = np.random.default_rng(1)
    f, _ = K.frequencies(32, 1e4)
    x, y = rng.standard_normal((2, 1, 1, 48))
    at = lambda v, p: K.rope(v, np.array([p]), f, interleaved)[0, 0]
    assert np.allclose(np.linalg.norm(at(x, 1234)), np.linalg.norm(x)) and np.array_equal(at(x, 77)[32:], x[0, 0, 32:])
    assert np.allclose(at(x, 900) @ at(y, 870), at(x, 30) @ at(y, 0))  # the distance alone counts
    quarter = K.rope(np.array([[[1.0, 0.0]]]), np.array([1]), np.array([np.pi / 2]), interleaved)
    assert np.allclose(quarter, [[[0, 1]]])


def test_norm_by_hand():
    y = K.rope(np.array([[[3.0, 4.0]]]), np.array([5]), np.zeros(0), norm=np.array([2.0, 1.0]), eps=0.0)
    assert np.allclose(y, np.array([[[6.0, 4.0]]]) / np.sqrt(12.5))


def test_frequencies():
    plain, one = K.frequencies(8, 1e4)
    assert np.allclose(plain, [1, 0.1, 0.01, 0.001]) and one == 1
    assert np.allclose(K.frequencies(8, 1e4, "linear", 4)[0], plain / 4)
    longer = K.frequencies(8, 1e4, "base", 8)[0]
    assert longer[0] == 1 and np.isclose(longer[-1], plain[-1] / 8)  # the slowest pair is factor times slower
    for kind in ("ramp", "waves"):
        f, _ = K.frequencies(128, 1e4, kind, 4, 1, 32, 4096)
        p, _ = K.frequencies(128, 1e4)
        turns = 4096 * p / (2 * np.pi)
        # the ramp's edges are whole pairs: one pair of room
        assert np.allclose(f[turns > 32 * 1.4], p[turns > 32 * 1.4]) and np.allclose(f[turns < 0.7], p[turns < 0.7] / 4)
        assert (np.diff(f) < 0).all()


@pytest.mark.parametrize("most", [2.0 ** -24, 1e-3, 1.0, 126.0, 127.0, 128.0, 65504.0])
def test_least_scale(most):
    most = float(np.float16(most))
    s = K.least_scale(most)
    fraction, _ = np.frexp(s)
    assert most <= 127 * s and fraction * 256 == int(fraction * 256)
    assert most > 127 * s * (1 - 2.0 ** -7)  # the next one down does not hold it


def test_write_read_by_hand():
    codes, scale = np.full((3, 1, 64, 64), 5), np.array([[1.0], [2.0], [0.0]])
    x = np.zeros((3, 1, 64))
    x[:, 0, 0] = [254.0, 3.0, 600.0]
    batch = (None, [66], np.array([[2, 1]]), 1, 3, 3)  # position 63 in page 2, 64 and 65 in page 1
    K.write(codes, scale, x, batch)
    assert scale[2, 0] == 2.0 and codes[2, 0, 63, 0] == 127  # scale 0: its own
    assert scale[1, 0] == 4.75 and codes[1, 0, 0, 0] == 1 and codes[1, 0, 1, 0] == 126  # begun anew
    assert (codes[1, 0, 2:] == 5).all()
    y = np.zeros((1, 1, 64))
    y[0, 0, 0] = 1300.0
    K.write(codes, scale, y, (None, [67], np.array([[2, 1]]), 1, 1, 1))
    assert scale[1, 0] == 19.0 and codes[1, 0, 1, 0] == 32 and codes[1, 0, 2, 0] == 68  # 126 / 4 = 31.5 to even
    back = K.read(codes, scale, (None, [67], np.array([[2, 1]]), 1, 2, 2))
    assert back[0, 0, 0] == 32 * 19 and back[1, 0, 0] == 68 * 19
    assert (K.read(codes, scale, (None, [1], np.array([[-1]]), 1, 1, 1)) == 0).all()


def test_attention_against_brute_force():
    rng = np.random.default_rng(2)
    kc, vc = rng.integers(-127, 128, (2, 4, 2, 64, 64))
    ks, vs = rng.uniform(0.001, 0.01, (2, 4, 2))
    q = rng.standard_normal((5, 4, 64))
    batch = (np.array([0, 3, 5]), [100, 1], np.array([[3, 0], [2, -1]]), 2, 5, 3)
    for window, causal in ((0, True), (9, True), (0, False)):
        y, size, _ = K.attention(kc, ks, vc, vs, q, batch, 0.125, window, causal)
        for r, s, at in ((0, 0, 97), (1, 0, 98), (2, 0, 99), (3, 1, -1), (4, 1, 0)):
            for h in range(4):
                num, den = np.zeros(64), 0.0
                for t in range([100, 1][s]):
                    if causal and (t > at or (window and t <= at - window)):
                        continue
                    p = batch[2][s][t // 64]
                    e = np.exp(0.125 * float((kc[p, h // 2, t % 64] * ks[p, h // 2]) @ q[r, h]))
                    num, den = num + e * vc[p, h // 2, t % 64] * vs[p, h // 2], den + e
                want = num / den if den else num
                assert np.allclose(y[r, h], want) and (size[r, h] >= np.abs(y[r, h]) - 1e-12).all()

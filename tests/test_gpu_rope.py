"""tern_rope on the GPU against the oracle: layouts, parts of a head, norms,
far positions, strides, in place."""
import numpy as np
import pytest
import torch

from gpu_util import say
from kv_util import TINY16, U16, U32, dev, half
from oracle import kv_oracle as K
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu

# sin and cos: a turn rounded to FP32 (2^-25 of a turn) and the instruction
# (2^-22.9 measured over every FP32 of half a turn)
TRIG = 2 * np.pi * 2.0 ** -25 + 2.0 ** -22.9


def bound(x, y, rot, amp, interleaved, norm, eps):
    """Of each value: the output's rounding; the pair's magnitude times the
    angle's error and four roundings; the norm's dim + 8 roundings."""
    n = np.abs(K.rope(x, np.zeros(len(x)), np.zeros(0), norm=norm, eps=eps))
    pair = n.copy()
    half_ = rot // 2
    for i in range(half_):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half_)
        both = (n[..., lo] + n[..., hi]) * amp
        pair[..., lo] = pair[..., hi] = both
    each = TRIG + 4 * U32 + (0 if norm is None else (x.shape[-1] + 8) * U32)
    return U16 * np.abs(y) + TINY16 + pair * each


def run(x, pos, rot, interleaved=False, amp=1.0, norm=None, eps=1e-6, base=1e6, **kw):
    freq, _ = K.frequencies(rot, base)
    rope = L.Rope(dev(freq), interleaved, amp, None if norm is None else dev(norm), eps)
    got = L.tern_rope(dev(x), dev(pos), rope, **kw)
    y = K.rope(x, pos, freq, interleaved, np.float64(np.float32(amp)), norm, np.float64(np.float32(eps)))
    off = np.abs(got.float().cpu().numpy() - y) / bound(x, y, rot, amp, interleaved, norm, eps)
    assert off.max() <= 1, f"{off.max():.3g} of the bound"
    return got


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("m,heads,dim,rot", [
    (1, 1, 8, 8), (1, 40, 128, 128), (3, 5, 64, 64), (7, 3, 64, 32), (2, 9, 96, 96), (5, 2, 80, 26), (4, 33, 128, 2), (6, 1, 256, 256),
    (2, 7, 512, 512), (700, 6, 128, 128), (513, 40, 64, 48), (33, 4, 24, 0), (9, 3, 120, 118), (17, 2, 128, 100), (600, 1, 16, 14)])
def test_rope(m, heads, dim, rot, interleaved):
    say("rope", m, heads, dim, rot, interleaved)
    rng = np.random.default_rng(m + heads + dim + rot)
    x = half(rng, m, heads, dim)
    pos = rng.integers(0, 5000, m).astype(np.int32)
    run(x, pos, rot, interleaved)
    run(x, pos, rot, interleaved, amp=1.25, norm=half(rng, dim), eps=1e-5)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    rng = np.random.default_rng(5)
    pos = np.array([0, 1, -1, 4095, 131072, 999999, 1 << 24, (1 << 24) + 1, (1 << 30) - 1, -(1 << 20), (1 << 31) - 1], np.int32)
    # angles beyond 2^53 / 1e6 turns are past what FP64 positions leave; the oracle's
    # own angle is rounded there: 2^31 * 2^-53 radians are far below TRIG
    run(half(rng, len(pos), 4, 128), pos, 128, interleaved)


@pytest.mark.parametrize("spread", [1e-6, 1e-3, 300.0])
def test_sizes_of_values(spread):
    """Subnormal and large values, with and without the norm; the norm of
    zeros."""
    rng = np.random.default_rng(7)
    x = half(rng, 5, 3, 128, spread=spread)
    x[2] = 0
    pos = np.arange(5, dtype=np.int32)
    run(x, pos, 128)
    run(x, pos, 64, norm=half(rng, 128), eps=1e-5)


def test_strides_and_in_place():
    rng = np.random.default_rng(9)
    rows = half(rng, 37, 20 * 64)
    freq, _ = K.frequencies(64, 1e4)
    rope = L.Rope(dev(freq))
    pos = np.arange(100, 137, dtype=np.int32)
    full = dev(rows)
    x = full.view(37, 20, 64)[:, 3:9]
    want = L.tern_rope(x.contiguous(), dev(pos), rope)
    assert torch.equal(L.tern_rope(x, dev(pos), rope), want)
    wide = torch.full((37, 11, 64), 7.0, dtype=torch.float16, device="cuda")
    L.tern_rope(x, dev(pos), rope, out=wide[:, 2:8])
    assert torch.equal(wide[:, 2:8], want) and (wide[:, :2] == 7).all() and (wide[:, 8:] == 7).all()
    L.tern_rope(x, dev(pos), rope, out=x)
    assert torch.equal(x, want)
    rest = torch.ones(20, dtype=torch.bool)
    rest[3:9] = False
    assert torch.equal(full.view(37, 20, 64)[:, rest], dev(rows).view(37, 20, 64)[:, rest])


def test_infinities_reach_their_own_head_alone():
    rng = np.random.default_rng(11)
    x = half(rng, 4, 5, 128)
    freq, _ = K.frequencies(128, 1e6)
    rope, pos = L.Rope(dev(freq), norm=dev(half(rng, 128))), dev(np.arange(4, dtype=np.int32))
    clean = L.tern_rope(dev(x), pos, rope)
    x[1, 2, 7], x[3, 0, 100] = np.nan, np.inf
    got = L.tern_rope(dev(x), pos, rope)
    other = torch.ones(4, 5, dtype=torch.bool)
    other[1, 2] = other[3, 0] = False
    assert torch.equal(got[other], clean[other]) and not torch.isfinite(got[1, 2]).any()


def test_empty():
    freq, _ = K.frequencies(64, 1e4)
    rope = L.Rope(dev(freq))
    assert L.tern_rope(torch.empty((0, 4, 64), dtype=torch.float16, device="cuda"), dev(np.zeros(0, np.int32)), rope).shape == (0, 4, 64)
    assert L.tern_rope(torch.empty((4, 0, 64), dtype=torch.float16, device="cuda"), dev(np.zeros(4, np.int32)), rope).numel() == 0

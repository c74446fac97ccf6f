"""tern_q4_gemm and tern_q4_experts on each of the tiles that they can take:
every group size, with and without zero points, more K steps than the two that
are staged, scales read four groups at a time and one by one, K that ends
inside a step.  Which tile a case takes is asserted."""
import numpy as np
import pytest

from gpu_util import say, to_dev
from oracle import q4_oracle as Q
from q4_util import activations, half, kind_of, upload, weights
from q4_util import check as check_rows
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu

# rows of the tile: m, n
WIDE = {32: (27, 49157), 64: (400, 4111), 96: (770, 6001), 128: (700, 9741)}
# k: groups a multiple of four or not; 5 to 8 K steps, the last one whole or not
LENGTHS = {32: (736, 1024), 64: (704, 1024), 128: (640, 1024)}


def wide(tile, group, zero, k, out):
    """All elements against FP64 products of the dequantized weights."""
    import torch
    say("wide", tile, group, zero, k, out)
    m, n = WIDE[tile]
    rng = np.random.default_rng(tile + group + k)
    w = upload(weights(rng, (), n, k, group, zero))
    x = half(activations(rng, m, k))
    assert L.load().tern_q4_tile_rows(w._at, m) == tile
    q = w.unpack().double().view(n, k // group, group)
    q = q - (8.0 if w.zero is None else w.zero.double().unsqueeze(-1))
    dense = (q * w.scale.double().unsqueeze(-1)).view(n, k).t().contiguous()
    y, b = x.double() @ dense, x.double().abs() @ dense.abs()
    half_step = 2.0 ** -11 if out == "f16" else 2.0 ** -24
    err = Q.adds(k, group) * Q.ADD * b
    tol = err + (y.abs() + err) * half_step + 2.0 ** -25
    got = L.tern_q4_gemm(w, x, kind_of(out))
    bad = ~((got.double() - y).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, e.g. {bad.nonzero()[:4].tolist()}"
    assert torch.equal(got, L.tern_q4_gemm(w, x, kind_of(out))), "two runs differ"


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("tile", list(WIDE))
def test_wide_tiles(tile, group, zero):
    for k, out in zip(LENGTHS[group], ("f32", "f16")):
        wide(tile, group, zero, k, out)


@pytest.mark.parametrize("m,n,k,group", [(400, 700, 3200, 64), (350, 40, 9728, 32), (1000, 130, 4096, 128)])
def test_tiles_in_k_parts(m, n, k, group):
    """Few tiles: K parts of many steps each, added by the reduction."""
    say("parts", m, n, k, group)
    rng = np.random.default_rng(m)
    w = weights(rng, (), n, k, group, True)
    wd, x = upload(w), activations(rng, m, k)
    assert L.load().tern_q4_tile_rows(wd._at, m) > 0 and L.load().tern_q4_workspace_bytes(wd._at, m) > 256
    y, _, err = Q.gemm(*w, group, x)
    check_rows(L.tern_q4_gemm(wd, half(x), L.TERN_F32), y, err, "f32", "K parts")


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group,hidden,inner", [(32, 736, 672), (64, 704, 1024), (128, 1024, 640)])
@pytest.mark.parametrize("rows", [0, 8, 16, 32, 64])
def test_experts_tiles(rows, group, hidden, inner, zero):
    """Some tokens of each route against the oracle."""
    say("experts", rows, group, hidden, inner, zero)
    m, topk, count = {0: (7, 2, 5), 8: (60, 2, 40), 16: (27, 2, 10), 32: (150, 2, 8), 64: (211, 2, 5)}[rows]
    if rows == 16 and group == 128:  # tiles of 16 rows end where 32 begin to pay: 5 rows an expert
        m = 26
    rng = np.random.default_rng(rows + group)
    up, down = weights(rng, (count,), 2 * inner, hidden, group, zero), weights(rng, (count,), 300, inner, group, zero)
    u, d = upload(up), upload(down)
    assert L.load().tern_q4_experts_tile_rows(u._at, d._at, m, topk) == rows
    x = activations(rng, m, hidden)
    ids = rng.integers(-1, count, (m, topk)).astype(np.int32)
    g = rng.uniform(0.01, 1, (m, topk)).astype(np.float32)
    got = L.tern_q4_experts(u, d, half(x), to_dev(ids), to_dev(g), L.TERN_F32)
    some = np.sort(rng.permutation(m)[:7])
    y, err = Q.experts(up, down, group, x[some], ids[some], g[some], parts=1 if rows else 2)
    check_rows(got[some], y, err, "f32", f"tiles of {rows}")
    assert (got == L.tern_q4_experts(u, d, half(x), to_dev(ids), to_dev(g), L.TERN_F32)).all(), "two runs differ"


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(20, 7200, 128), (32, 12293, 896), (77, 2561, 1664), (77, 2561, 1792), (130, 1700, 512)])
def test_short_rows_of_some_tens_of_activations(m, n, k, group, zero):
    """Few K tiles for the wavefronts that share them: on both sides of the rule."""
    say("short", m, n, k, group, zero)
    rng = np.random.default_rng(m + k)
    w = weights(rng, (), n, k, group, zero)
    wd, x = upload(w), activations(rng, m, k)
    assert L.load().tern_q4_tile_rows(wd._at, m) == 0
    y, _, err = Q.gemm(*w, group, x)
    for out in ("f32", "f16"):
        check_rows(L.tern_q4_gemm(wd, half(x), kind_of(out)), y, err, out, "short rows")


def far_codes(n, k, group):
    """Random codes of over 16 GiB, and rows of them as the oracle takes them."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    codes = torch.empty((n, k // 2), dtype=torch.uint8, device="cuda")
    for part in codes.chunk(16):
        part.random_(0, 256, generator=gen)
    scale = torch.rand((n, k // group), device="cuda", generator=gen).half()
    pick = [0, 1, n // 2, n - 18, n - 1]
    q = np.stack([L.Q4Matrix(codes[r:r + 1].clone(), scale[r:r + 1].clone()).unpack().cpu().numpy()[0] for r in pick])
    return codes, scale, pick, (q, scale[pick].cpu().numpy(), None)


def test_product_past_the_tiles_buffers():
    """So many scales that a prefill batch runs on the kernel for few rows."""
    import torch
    n, k, m = (1 << 20) + 3, 32768, 330
    say("far scales", n, k, m)
    codes, scale, pick, rows = far_codes(n, k, 128)
    w = L.Q4Matrix(codes, scale)
    assert L.load().tern_q4_tile_rows(w._at, m) == 0
    x = activations(np.random.default_rng(1), m, k)
    y, _, err = Q.gemm(*rows, 128, x)
    got = L.tern_q4_gemm(w, half(x), L.TERN_F32)
    check_rows(got[:, pick], y, err, "f32", "far scales")
    del codes, scale, w, got
    torch.cuda.empty_cache()


def test_experts_past_the_tiles_buffers():
    """The same of an expert's down product: tiles of 16 rows."""
    import torch
    n, k, m = (1 << 15) + 5, 1 << 20, 70
    say("far scales of an expert", n, k, m)
    rng = np.random.default_rng(2)
    codes, scale, pick, rows = far_codes(n, k, 128)
    up = weights(rng, (1,), 2 * k, 32, 32, False)
    u, d = upload(up), L.Q4Matrix(codes.unsqueeze(0), scale.unsqueeze(0))
    assert L.load().tern_q4_experts_tile_rows(u._at, d._at, m, 1) == 16
    x = rng.standard_normal((m, 32)).astype(np.float16)
    ids, g = np.zeros((m, 1), np.int32), np.ones((m, 1), np.float32)
    got = L.tern_q4_experts(u, d, half(x), to_dev(ids), to_dev(g), L.TERN_F32)
    some = [0, m - 1]
    q, s = (t[None] for t in rows[:2])
    y, err = oracle_groups(up, (q, s, None), x[some])
    check_rows(got[some][:, pick], y, err, "f32", "far scales of an expert")
    del codes, scale, d, got
    torch.cuda.empty_cache()


def oracle_groups(up, down, x):
    """Q.experts with groups of 32 in gate and up, 128 in down: the finer
    groups' scales repeat the coarser ones'."""
    q, s, z = down
    y, err = Q.experts(up, (q, np.repeat(s, 4, axis=-1), z), 32, x, np.zeros((len(x), 1), np.int32), np.ones((len(x), 1), np.float32))
    return y, err

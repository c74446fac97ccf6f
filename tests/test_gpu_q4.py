"""tern_q4_gemm, tern_q4_pack and tern_q4_unpack on the GPU against the
oracle: every route (rows and tiles, K parts), group size, zero points, odd
sizes, values out of the ordinary."""
import numpy as np
import pytest

from gpu_util import say, to_dev
from oracle import q4_oracle as Q
from q4_util import activations, check, half, kind_of, replay_checks, upload, weights
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu

SHAPES = [
    # m, n, k in groups of 128
    (1, 16, 1), (1, 1, 1), (1, 257, 9), (2, 48, 2), (3, 100, 33), (15, 31, 5), (16, 64, 8), (17, 33, 3), (32, 130, 4),
    (33, 65, 7), (48, 16, 17), (64, 129, 2), (65, 127, 1), (65, 300, 9), (128, 128, 8), (129, 257, 3), (300, 140, 20),
    (70, 3, 96), (321, 129, 8), (400, 700, 17), (330, 33, 40), (513, 4400, 1), (2050, 4097, 2),
]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,kg", SHAPES)
def test_gemm_matches_oracle(m, n, kg, group):
    say("q4 gemm", m, n, kg, group)
    rng = np.random.default_rng(m * 1000 + n + group)
    # group 32: k ends inside a K step of 128 as often as not
    k = kg * 128 if group == 128 else max(group, kg * 128 - group * (n % 3))
    w = weights(rng, (), n, k, group, zero=(m + n) % 2 == 0)
    x = activations(rng, m, k)
    wd, xd = upload(w), half(x)
    y, _, err = Q.gemm(*w, group, x)
    for out in ("f16", "f32"):
        got = L.tern_q4_gemm(wd, xd, kind_of(out))
        check(got, y, err, out, f"{m}x{n}x{k} group {group} {out}")
        again = L.tern_q4_gemm(wd, xd, kind_of(out))
        assert (got == again).all(), "two runs differ"


@pytest.mark.parametrize("m,n,k,group,zero", [
    (1, 40, 20512, 32, True), (3, 9000, 2560, 32, True), (4, 32773, 64, 64, False), (2, 33000, 1280, 32, True),
    (13, 33000, 320, 64, True), (20, 28700, 96, 32, False), (40, 4100, 10240, 32, True), (31, 49300, 64, 64, True),
    (12, 40, 20512, 32, True), (20, 40, 20512, 32, True), (160, 1640, 10240, 32, True), (33, 70, 33024, 128, False)])
def test_gemm_long_rows_and_many_panels(m, n, k, group, zero):
    """Rows whose scales are staged in parts, and as many panels as change
    the kernel's shape."""
    say("q4 gemm", m, n, k, group)
    rng = np.random.default_rng(n + k)
    w = weights(rng, (), n, k, group, zero)
    x = activations(rng, m, k)
    y, _, err = Q.gemm(*w, group, x)
    check(L.tern_q4_gemm(upload(w), half(x), L.TERN_F32), y, err, "f32", f"{m}x{n}x{k} group {group}")


@pytest.mark.parametrize("m,n", [(700, 9728), (1500, 4096), (900, 5120), (512, 12300)])
def test_gemm_tile_sizes(m, n):
    """Each output tile of the tile kernel, by the sizes that choose it."""
    say("q4 gemm", m, n)
    rng = np.random.default_rng(m)
    w = weights(rng, (), n, 192, 64, True)
    x = activations(rng, m, 192)
    y, _, err = Q.gemm(*w, 64, x)
    check(L.tern_q4_gemm(upload(w), half(x), L.TERN_F32), y, err, "f32", f"{m}x{n}")


@pytest.mark.parametrize("m", [1, 20, 400])
def test_gemm_scales_and_zero_points_of_any_size(m):
    """Scales from subnormal to 60000 and zero points up to 255: FP32 outputs
    keep their precision and their range."""
    rng = np.random.default_rng(5)
    n, k, group = 70, 256, 64
    q, s, z = weights(rng, (), n, k, group, True, zmax=256)
    s[0::3] = np.float16(6e-8) * rng.integers(1, 900, s[0::3].shape)
    s[1::3] = rng.uniform(30000, 60000, s[1::3].shape).astype(np.float16)
    x = activations(rng, m, k)
    y, _, err = Q.gemm(q, s, z, group, x)
    check(L.tern_q4_gemm(upload((q, s, z)), half(x), L.TERN_F32), y, err, "f32", "wide scales")


@pytest.mark.parametrize("m", [3, 40, 400])
@pytest.mark.parametrize("group", [32, 128])
def test_gemm_bad_rows_and_scales_stay_alone(m, group):
    """A NaN or infinity in a row of x reaches that row of y alone, one in a
    weight row's scale that column; the rest equals the clean result."""
    import torch
    rng = np.random.default_rng(6)
    n, k = 90, 384 - 32 * (group == 32)
    w = weights(rng, (), n, k, group, True)
    x = activations(rng, m, k)
    wd = upload(w)
    clean = L.tern_q4_gemm(wd, half(x), L.TERN_F32)
    xb = x.copy()
    xb[1, 5], xb[2, k - 1] = np.nan, np.inf
    got = L.tern_q4_gemm(wd, half(xb), L.TERN_F32)
    rest = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(got[rest], clean[rest])
    assert got[1].isnan().all() and not got[2].isfinite().any()
    s = w[1].copy()
    s[4, 0], s[5, -1] = np.nan, np.inf
    got = L.tern_q4_gemm(upload((w[0], s, w[2])), half(x), L.TERN_F32)
    rest = [i for i in range(n) if i not in (4, 5)]
    assert torch.equal(got[:, rest], clean[:, rest])
    assert got[:, 4].isnan().all() and not got[:, 5].isfinite().any()


@pytest.mark.parametrize("m", [1, 33, 400])
def test_gemm_writes_its_output_alone(m):
    import torch
    rng = np.random.default_rng(7)
    n, k = 45, 160
    w = upload(weights(rng, (), n, k, 32, False))
    x = half(activations(rng, m, k))
    buf = torch.full((m + 2, n), -7.0, device="cuda")
    need = L.load().tern_q4_workspace_bytes(w._at, m)
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    L.tern_q4_gemm(w, x, L.TERN_F32, out=buf[1:-1], ws=ws[:need])
    assert (buf[0] == -7).all() and (buf[-1] == -7).all() and (buf[1:-1] != -7).all()
    assert (ws[need:] == 77).all()


@pytest.mark.parametrize("m", [0, 1, 400])
def test_gemm_empty(m):
    import torch
    w = L.Q4Matrix(torch.empty((5, 0), dtype=torch.uint8, device="cuda"), torch.empty((5, 0), dtype=torch.float16, device="cuda"))
    y = L.tern_q4_gemm(w, torch.empty((m, 0), dtype=torch.float16, device="cuda"), out=torch.ones((m, 5), dtype=torch.float16, device="cuda"))
    assert y.shape == (m, 5) and (y == 0).all()
    w = L.Q4Matrix(torch.empty((0, 64), dtype=torch.uint8, device="cuda"), torch.empty((0, 1), dtype=torch.float16, device="cuda"))
    assert L.tern_q4_gemm(w, torch.ones((m, 128), dtype=torch.float16, device="cuda")).shape == (m, 0)


@pytest.mark.parametrize("m", [1, 48, 400])
def test_gemm_captured_and_on_another_stream(m):
    import torch
    rng = np.random.default_rng(8)
    n, k = 200, 2048
    wd = upload(weights(rng, (), n, k, 64, True))
    x = half(activations(rng, m, k))
    y = torch.empty((m, n), dtype=torch.float16, device="cuda")
    ws = L.tern_q4_workspace(wd, m)
    replay_checks(lambda s: L.tern_q4_gemm(wd, x, out=y, stream=s, ws=ws),
                  lambda r: x.copy_(half(activations(rng, m, k))), [y])
    want = L.tern_q4_gemm(wd, x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):  # workspace and output allocated for the side stream
        got = L.tern_q4_gemm(wd, x, stream=side.cuda_stream)
        torch.full((1 << 20,), 3.0, device="cuda")
        side.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("m,n,k", [(40, 3600, 640), (64, 9000, 320), (30, 49300, 64)])
def test_gemm_captured_on_the_wide_kernels(m, n, k):
    """Workgroups of over 64 KiB of LDS, four panels, 32-row tiles."""
    import torch
    rng = np.random.default_rng(12)
    wd = upload(weights(rng, (), n, k, 64, False))
    x = half(activations(rng, m, k))
    y = torch.empty((m, n), device="cuda")
    ws = L.tern_q4_workspace(wd, m)
    replay_checks(lambda s: L.tern_q4_gemm(wd, x, L.TERN_F32, out=y, stream=s, ws=ws),
                  lambda r: x.copy_(half(activations(rng, m, k))), [y])


def test_gemm_offsets_past_32_bits():
    """Codes of over 4 GiB: rows at both ends against the oracle."""
    import torch
    rng = np.random.default_rng(9)
    n, k, group = (1 << 20) + 3, 8320, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scale = torch.rand((n, k // group), device="cuda", generator=gen).half()
    w = L.Q4Matrix(codes, scale)
    pick = [0, 1, n // 2, n - 20, n - 2, n - 1]
    q = np.stack([L.Q4Matrix(codes[r:r + 1].clone(), scale[r:r + 1].clone()).unpack().cpu().numpy()[0] for r in pick])
    s = scale[pick].cpu().numpy()
    for m in (1, 66, 170):
        x = activations(rng, m, k)
        y, _, err = Q.gemm(q, s, None, group, x)
        got = L.tern_q4_gemm(w, half(x), L.TERN_F32)
        check(got[:, pick], y, err, "f32", f"far rows, m={m}")


@pytest.mark.parametrize("shape", [(1, 8, 32), (3, 7, 96), (33, 4096)])
def test_pack_and_unpack(shape):
    import torch
    rng = np.random.default_rng(10)
    q = rng.integers(0, 16, shape, dtype=np.uint8)
    scale = torch.ones((*shape[:-1], shape[-1] // 32), dtype=torch.float16, device="cuda")
    w = L.Q4Matrix.from_codes(to_dev(q), scale)
    assert np.array_equal(w.codes.cpu().numpy(), Q.pack(q))
    assert np.array_equal(w.unpack().cpu().numpy(), q)
    q.reshape(-1)[-1] = 16
    with pytest.raises(L.TernError) as e:
        L.Q4Matrix.from_codes(to_dev(q), scale)
    assert e.value.status == L.TERN_E_INVAL


def test_gemm_refusals_of_tensors():
    import torch
    dev = dict(device="cuda")
    w = L.Q4Matrix(torch.zeros((8, 64), dtype=torch.uint8, **dev), torch.ones((8, 1), dtype=torch.float16, **dev))
    x = torch.ones((2, 128), dtype=torch.float16, **dev)
    for bad in (x.float(), x.cpu(), x[:, :64], torch.ones((128, 2), dtype=torch.float16, **dev).t(), x[0]):
        with pytest.raises(ValueError):
            L.tern_q4_gemm(w, bad)
    with pytest.raises(ValueError):
        L.tern_q4_gemm(w, x, out=torch.empty((2, 8), **dev))
    for ws in (torch.empty(1024, dtype=torch.uint8), torch.empty(2048, dtype=torch.uint8, **dev)[::2]):
        with pytest.raises(ValueError):
            L.tern_q4_gemm(w, x, ws=ws)
    with pytest.raises(ValueError):
        L.tern_q4_gemm(w, x, 7)
    with pytest.raises(L.TernError) as e:
        L.tern_q4_gemm(w, torch.ones(2 * 128 + 1, dtype=torch.float16, **dev)[1:].view(2, 128))
    assert e.value.status == L.TERN_E_ALIGN
    with pytest.raises(L.TernError) as e:
        big = torch.ones((400, 4096), dtype=torch.float16, **dev)
        wide = L.Q4Matrix(torch.zeros((8, 2048), dtype=torch.uint8, **dev), torch.ones((8, 32), dtype=torch.float16, **dev))
        L.tern_q4_gemm(wide, big, ws=torch.empty(16, dtype=torch.uint8, **dev))
    assert e.value.status == L.TERN_E_WORKSPACE
    with pytest.raises(ValueError):
        L.Q4Matrix(torch.zeros((8, 64), dtype=torch.uint8, **dev), torch.ones((7, 1), dtype=torch.float16, **dev))
    with pytest.raises(L.TernError):  # a group of 16
        L.Q4Matrix(torch.zeros((8, 64), dtype=torch.uint8, **dev), torch.ones((8, 8), dtype=torch.float16, **dev))

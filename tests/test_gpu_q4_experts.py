"""tern_q4_experts on the GPU against the oracle, on each of its routes (slot
by slot, tiles of 16, 32 and 64 rows), and with tern_route before it."""
import numpy as np
import pytest

from gpu_util import say, to_dev
from oracle import q4_oracle as Q
from q4_util import activations, check, half, kind_of, replay_checks, upload, weights
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu


def layer(rng, count, hidden, inner, width, group, zero):
    return (weights(rng, (count,), 2 * inner, hidden, group, zero), weights(rng, (count,), width, inner, group, zero))


def slots(rng, m, topk, count):
    ids = np.stack([rng.permutation(max(count, topk))[:topk] for _ in range(m)]).astype(np.int32) % count
    return ids, rng.uniform(0.01, 1, (m, topk)).astype(np.float32)


def compare(up, down, group, x, ids, g, what, outs=("f16", "f32")):
    y, err = Q.experts(up, down, group, x, ids, g)
    u, d = upload(up), upload(down)
    for out in outs:
        got = L.tern_q4_experts(u, d, half(x), to_dev(ids), to_dev(g), kind_of(out))
        check(got, y, err, out, f"{what} {out}")
        again = L.tern_q4_experts(u, d, half(x), to_dev(ids), to_dev(g), kind_of(out))
        assert (got == again).all(), "two runs differ"


# m, topk, experts, hidden, inner, width (in groups of 32, 64 or 128; width in rows)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,topk,count,hidden,inner,width", [
    (1, 1, 1, 1, 1, 1), (1, 8, 16, 3, 2, 130), (4, 8, 8, 5, 1, 33), (1, 2, 60, 2, 3, 65),     # slot by slot
    (11, 3, 20, 3, 2, 100), (25, 8, 100, 1, 1, 16),                                            # tiles of 16 rows
    (11, 3, 5, 3, 2, 100), (40, 2, 8, 2, 5, 47),
    (60, 2, 7, 3, 3, 129), (50, 1, 3, 5, 1, 20),
    (70, 2, 7, 2, 2, 130), (36, 3, 3, 5, 3, 129),                                              # of 32
    (150, 1, 2, 2, 1, 70), (130, 4, 4, 1, 3, 260),                                             # of 64
    (900, 1, 2, 2, 1, 70), (170, 5, 2, 4, 3, 300), (1100, 2, 30, 1, 1, 65),                                             # several an expert
])
def test_experts_match_oracle(m, topk, count, hidden, inner, width, group):
    say("experts", m, topk, count, hidden, inner, width, group)
    rng = np.random.default_rng(m * 100 + group)
    up, down = layer(rng, count, hidden * group, inner * group, width, group, zero=m % 2 == 0)
    ids, g = slots(rng, m, topk, count)
    compare(up, down, group, activations(rng, m, hidden * group), ids, g, "experts")


@pytest.mark.parametrize("m,topk,count,hidden,inner,width", [
    (1, 32, 8, 64, 384, 20), (2, 16, 8, 10240, 1024, 17), (1, 1, 1, 20480, 32, 5),              # slot by slot
    (30, 2, 20, 10240, 64, 18), (30, 2, 20, 64, 8192, 18), (70, 1, 64, 32, 10240, 40)])         # tiles of 16 rows
def test_experts_long_rows(m, topk, count, hidden, inner, width):
    """Rows whose scales are staged in parts."""
    say("experts", m, topk, count, hidden, inner, width)
    rng = np.random.default_rng(hidden + inner)
    up, down = layer(rng, count, hidden, inner, width, 32, True)
    ids, g = slots(rng, m, topk, count)
    # small activations: the inner values stay in FP16's range
    x = (activations(rng, m, hidden).astype(np.float64) / 64).astype(np.float16)
    compare(up, down, 32, x, ids, g, "long rows", outs=("f32",))


def test_experts_of_more_slots_than_a_round():
    """Tokens in several rounds: the same rows as calls on parts of them, and
    the oracle's at the rounds' ends."""
    import torch
    rng = np.random.default_rng(11)
    m, topk, count = (1 << 19) + 1000, 2, 3
    up, down = layer(rng, count, 32, 32, 8, 32, False)
    u, d = upload(up), upload(down)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((m, 32), device="cuda", generator=gen).half()
    ids = torch.randint(-1, count, (m, topk), device="cuda", generator=gen, dtype=torch.int32)
    g = torch.rand((m, topk), device="cuda", generator=gen)
    got = L.tern_q4_experts(u, d, x, ids, g, L.TERN_F32)
    edge = 1 << 18
    for a, b in ((0, 40), (edge - 300, edge + 300), (2 * edge - 5, 2 * edge + 11), (m - 1000, m)):
        part = L.tern_q4_experts(u, d, x[a:b], ids[a:b].contiguous(), g[a:b].contiguous(), L.TERN_F32)
        if (b - a) * topk > 32:
            assert torch.equal(got[a:b], part)
        else:  # slot by slot: gates go into the FP32 sums, in another order than on tiles, so both meet the oracle
            y, err = Q.experts(up, down, 32, x[a:b].cpu().numpy(), ids[a:b].cpu().numpy(), g[a:b].cpu().numpy())
            check(got[a:b], y, err, "f32", "tiles")
            check(part, y, err, "f32", "slot by slot")
    for a in (0, edge - 8, 2 * edge - 8, m - 16):
        part = slice(a, a + 16)
        y, err = Q.experts(up, down, 32, x[part].cpu().numpy(), ids[part].cpu().numpy(), g[part].cpu().numpy())
        check(got[part], y, err, "f32", f"tokens from {a}")


@pytest.mark.parametrize("m,topk,count", [(3, 4, 4), (20, 2, 20), (30, 2, 8), (60, 2, 4), (150, 2, 4), (600, 2, 3)])
def test_experts_skipped_repeated_and_lopsided(m, topk, count):
    """Ids outside the range, tokens with none, one expert for all, the same
    expert twice."""
    rng = np.random.default_rng(4)
    up, down = layer(rng, count, 64, 96, 40, 32, True)
    x = activations(rng, m, 64)
    ids, g = slots(rng, m, topk, count)
    ids[rng.random(ids.shape) < 0.3] = -1
    ids[0] = [count, 2 ** 31 - 1, -2 ** 31, -5][:topk]
    compare(up, down, 32, x, ids, g, "skipped")
    one = np.full_like(ids, count - 1)
    compare(up, down, 32, x, one, g, "one expert", outs=("f32",))
    none = np.full_like(ids, -1)
    got = L.tern_q4_experts(upload(up), upload(down), half(x), to_dev(none), to_dev(g))
    assert (got == 0).all()


@pytest.mark.parametrize("m,topk,count,hidden,inner,group", [
    (1, 1, 4, 256, 128, 128), (1, 8, 64, 2560, 1024, 128), (4, 8, 8, 320, 96, 32), (32, 1, 5, 128, 64, 64)])
def test_few_slots_keep_their_inner_values(m, topk, count, hidden, inner, group):
    """Up to 32 slots the inner values come as two FP16 values each: the bound
    has their rounding squared."""
    rng = np.random.default_rng(15)
    up, down = layer(rng, count, hidden, inner, 40, group, True)
    ids, g = slots(rng, m, topk, count)
    x = (activations(rng, m, hidden).astype(np.float64) / 16).astype(np.float16)
    y, err = Q.experts(up, down, group, x, ids, g, parts=2)
    check(L.tern_q4_experts(upload(up), upload(down), half(x), to_dev(ids), to_dev(g), L.TERN_F32), y, err, "f32", "few slots")


def test_few_slots_past_fp16_are_infinite():
    """An inner value beyond FP16 is infinite, its rest nothing: no NaN."""
    import torch
    rng = np.random.default_rng(16)
    up, down = layer(rng, 1, 64, 32, 3, 32, False)
    q = np.full_like(up[0], 15)
    up = (q, np.full_like(up[1], np.float16(4.0)), None)
    down = (np.full_like(down[0], 9), np.ones_like(down[1]), None)  # weights 1
    x = half(np.ones((1, 64), np.float16))
    got = L.tern_q4_experts(upload(up), upload(down), x, to_dev(np.zeros((1, 1), np.int32)), to_dev(np.ones((1, 1), np.float32)),
                            L.TERN_F32)
    assert torch.isinf(got).all() and (got > 0).all()


def test_experts_bad_rows_stay_alone():
    import torch
    rng = np.random.default_rng(5)
    for m, count in ((3, 4), (30, 20), (30, 8), (120, 2), (420, 2)):
        up, down = (upload(w) for w in layer(rng, count, 128, 64, 50, 64, False))
        x = activations(rng, m, 128)
        ids, g = slots(rng, m, 2, count)
        clean = L.tern_q4_experts(up, down, half(x), to_dev(ids), to_dev(g))
        x[1, 3] = np.nan
        got = L.tern_q4_experts(up, down, half(x), to_dev(ids), to_dev(g))
        rest = [i for i in range(m) if i != 1]
        assert torch.equal(got[rest], clean[rest]) and got[1].isnan().all()


def test_experts_write_their_output_alone():
    import torch
    rng = np.random.default_rng(6)
    for m, count in ((2, 4), (30, 20), (30, 8), (120, 2), (420, 2)):
        up, down = (upload(w) for w in layer(rng, count, 64, 32, 33, 32, False))
        ids, g = slots(rng, m, 2, count)
        buf = torch.full((m + 2, 33), -7.0, dtype=torch.float16, device="cuda")
        need = L.load().tern_q4_experts_workspace_bytes(up._at, down._at, m, 2)
        ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
        L.tern_q4_experts(up, down, half(activations(rng, m, 64)), to_dev(ids), to_dev(g), out=buf[1:-1], ws=ws[:need])
        assert (buf[0] == -7).all() and (buf[-1] == -7).all() and (buf[1:-1] != -7).all() and (ws[need:] == 77).all()


def test_experts_empty():
    import torch
    rng = np.random.default_rng(7)
    up, down = (upload(w) for w in layer(rng, 4, 64, 32, 33, 32, False))
    i, f = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float32, device="cuda")
    h = dict(dtype=torch.float16, device="cuda")
    assert L.tern_q4_experts(up, down, torch.empty((0, 64), **h), torch.empty((0, 2), **i), torch.empty((0, 2), **f)).shape == (0, 33)
    bare = L.Q4Matrix(torch.empty((4, 64, 0), dtype=torch.uint8, device="cuda"), torch.empty((4, 64, 0), **h))
    for m in (2, 40, 300):  # no inputs: nothing to multiply
        ids, g = torch.zeros((m, 2), **i), torch.ones((m, 2), **f)
        assert (L.tern_q4_experts(bare, down, torch.empty((m, 0), **h), ids, g) == 0).all()


@pytest.mark.parametrize("m,topk,count", [(1, 4, 8), (30, 4, 8), (300, 2, 4)])
def test_routed_layer_captured(m, topk, count):
    """Routing and experts together, as a decode step calls them, eager and in
    a graph, against the oracle's two in a row."""
    import torch
    rng = np.random.default_rng(8)
    up, down = layer(rng, count, 128, 64, 72, 64, True)
    bias = (0.1 * rng.standard_normal(count)).astype(np.float32)
    opts = dict(groups=2, group_best=2, keep_groups=2, renorm=True, scale=1.5)
    e = L.Q4Experts(upload(up), upload(down), topk, score=L.TERN_SCORE_SIGMOID, bias=to_dev(bias), **opts)
    x, l = half(activations(rng, m, 128)), to_dev(rng.standard_normal((m, count)).astype(np.float32))
    y = torch.empty((m, 72), device="cuda")
    ws = L.tern_q4_experts_workspace(e.gate_up, e.down, m, topk)
    ids = torch.empty((m, topk), dtype=torch.int32, device="cuda")
    g = torch.empty((m, topk), device="cuda")

    def call(stream):
        L.tern_route(l, topk, L.TERN_SCORE_SIGMOID, e._route["bias"], ids=ids, weights=g, stream=stream, **opts)
        L.tern_q4_experts(e.gate_up, e.down, x, ids, g, L.TERN_F32, out=y, stream=stream, ws=ws)

    def change(rep):
        x.copy_(half(activations(rng, m, 128)))
        l.normal_()

    replay_checks(call, change, [y, ids, g])
    side = torch.cuda.Stream()
    for stream in (None, side.cuda_stream):
        got = e.run(x, l, L.TERN_F32, stream=stream)
        side.synchronize()
        assert torch.equal(got, y)
    want, weight = Q.route(l.cpu().numpy(), topk, "sigmoid", bias, 2, 2, 2, True, 1.5)
    assert np.array_equal(ids.cpu().numpy(), want)
    xs = x.cpu().numpy()
    out, err = Q.experts(up, down, 64, xs, want, weight.astype(np.float32))
    # the weights' own half step
    check(y, out, err + 2.0 ** -23 * np.abs(out), "f32", "routed layer")


@pytest.mark.parametrize("m,count", [(2, 4), (30, 20), (60, 8), (150, 4)])
def test_skipped_slots_weights_are_not_looked_at(m, count):
    import torch
    rng = np.random.default_rng(13)
    up, down = (upload(w) for w in layer(rng, count, 64, 32, 33, 32, False))
    x = half(activations(rng, m, 64))
    ids, g = slots(rng, m, 2, count)
    ids[::2, 1] = -1
    g[::2, 1] = 0.5
    want = L.tern_q4_experts(up, down, x, to_dev(ids), to_dev(g))
    g[::4, 1], g[2::4, 1] = np.nan, np.inf
    assert torch.equal(L.tern_q4_experts(up, down, x, to_dev(ids), to_dev(g)), want) and want.isfinite().all()


@pytest.mark.parametrize("m,topk,count", [(1, 4, 8), (30, 4, 16), (100, 2, 4)])
def test_layer_captured_with_its_own_buffers(m, topk, count):
    """Q4Experts.run and tern_q4_gemm in a graph, their outputs and workspaces
    from the graph's pool; another graph of the same layer beside it."""
    import torch
    rng = np.random.default_rng(14)
    up, down = (upload(w) for w in layer(rng, count, 128, 64, 72, 64, False))
    head = upload(weights(rng, (), 200, 128, 64, True))
    e = L.Q4Experts(up, down, topk)
    x, l = half(activations(rng, m, 128)), to_dev(rng.standard_normal((m, count)).astype(np.float32))
    big = half(activations(rng, 400, 128))

    def step():
        return e.run(x, l), L.tern_q4_gemm(head, big)

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step())
    for _ in range(3):
        x.copy_(half(activations(rng, m, 128)))
        l.normal_()
        want = step()
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_two_calls_at_once_on_two_streams():
    import torch
    rng = np.random.default_rng(9)
    up, down = (upload(w) for w in layer(rng, 8, 256, 128, 96, 64, False))
    streams = [torch.cuda.Stream() for _ in range(2)]
    args, want = [], []
    for i in range(2):
        ids, g = slots(rng, 60, 2, 8)
        args.append((half(activations(rng, 60, 256)), to_dev(ids), to_dev(g)))
        want.append(L.tern_q4_experts(up, down, *args[i]))
    torch.cuda.synchronize()
    for _ in range(10):
        got = [L.tern_q4_experts(up, down, *args[i], stream=streams[i].cuda_stream) for i in range(2)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_experts_refusals_of_tensors():
    import torch
    rng = np.random.default_rng(10)
    up, down = (upload(w) for w in layer(rng, 4, 64, 32, 33, 32, False))
    x = half(activations(rng, 3, 64))
    ids, g = (to_dev(a) for a in slots(rng, 3, 2, 4))
    call = lambda **kw: L.tern_q4_experts(**{**dict(gate_up=up, down=down, x=x, ids=ids, weights=g), **kw})
    for kw in (dict(x=x[:, :32]), dict(x=x[:2]), dict(ids=ids.long()), dict(ids=ids.t().contiguous()), dict(ids=ids.cpu()),
               dict(weights=g[:, :1]), dict(weights=g.half()), dict(ws=torch.empty(1 << 20, dtype=torch.uint8)), dict(out=torch.empty((3, 33), device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(down=up), dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(L.TernError):
            call(**kw)
    e = L.Q4Experts(up, down, 2)
    with pytest.raises(ValueError):
        e.run(x, torch.zeros((3, 5), device="cuda"))

"""Positions, cache and attention as a program uses them: a decoder layer's
attention block with packed projections, prompt and tokens; captured and
replayed calls; streams; two calls at once; refusals of the binding."""
import threading
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import check_y, oracle_y, small_matrix, upload_pack
from kv_util import Case, check_attention, dev, half
from oracle import kv_oracle as K
from q4_util import replay_checks
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM = 256, 4, 2, 64


class Layer:
    """q, k, v and o projections of packed trits; norms of the heads; a cache."""

    def __init__(self, rng, pages):
        shapes = ((HEADS * DIM, HIDDEN), (KV * DIM, HIDDEN), (KV * DIM, HIDDEN), (HIDDEN, HEADS * DIM))
        self.mats = [small_matrix(n, k, 64, 1, 0.0, seed=90 + i)[0] for i, (n, k) in enumerate(shapes)]
        for m in self.mats:
            m["scales"] *= np.float16(0.25)
        self.packed = [upload_pack(m, O.FMT_2BIT) for m in self.mats]
        self.freq, _ = K.frequencies(DIM, 1e4)
        self.norms = [(1 + 0.1 * rng.standard_normal(DIM)).astype(np.float16) for _ in range(2)]
        self.rope = [L.Rope(dev(self.freq), norm=dev(n)) for n in self.norms]
        self.cache = L.KvCache.empty(pages, KV, DIM)

    def plan(self, x):
        """The buffers and plans for x's number of rows."""
        m = x.shape[0]
        new = lambda n: torch.empty((m, n), dtype=torch.float16, device="cuda")
        q, k, v, out = new(HEADS * DIM), new(KV * DIM), new(KV * DIM), new(HIDDEN)
        y = new(HEADS * DIM)
        return L.Plan(self.packed[:3], [x] * 3, [q, k, v]), L.Plan(self.packed[3:], [y], [out]), (q, k, v, y, out)

    def run(self, plans, batch, stream=None, ws=None):
        before, after, (q, k, v, y, out) = plans
        m = q.shape[0]
        before.run(stream)
        turned = L.tern_kv_write(self.cache, batch, k.view(m, KV, DIM), v.view(m, KV, DIM), rope=self.rope[1],
                                 q=q.view(m, HEADS, DIM), q_rope=self.rope[0], stream=stream)
        L.tern_kv_attention(self.cache, batch, turned, out=y.view(m, HEADS, DIM), stream=stream, ws=ws)
        after.run(stream)
        return turned


def check_block(layer, twin, plans, x, pos, host, batch):
    """Every step against its own oracle: the products' bound, the turned rows
    and the cache's bytes equal to those of separate calls, the attention over
    the cache as it is, the last product."""
    q, k, v, y, out = plans[2]
    m = len(x)
    turned = layer.run(plans, batch)
    for got, mat, given in ((q, layer.mats[0], x), (k, layer.mats[1], x), (v, layer.mats[2], x)):
        check_y(got, *oracle_y(mat, given), "projection")
    assert torch.equal(turned, L.tern_rope(q.view(m, HEADS, DIM), dev(pos), layer.rope[0]))
    L.tern_kv_write(twin, batch, L.tern_rope(k.view(m, KV, DIM), dev(pos), layer.rope[1]), v.view(m, KV, DIM))
    own = layer.cache
    for a, b in ((own.k, twin.k), (own.v, twin.v), (own.k_scale, twin.k_scale), (own.v_scale, twin.v_scale)):
        assert torch.equal(a, b)
    codes = [K.unpack(t.cpu().numpy(), DIM, keys) for t, keys in ((own.k, True), (own.v, False))]
    c = SimpleNamespace(kc=codes[0], vc=codes[1], ks=own.k_scale.cpu().numpy().astype(np.float64),
                        vs=own.v_scale.cpu().numpy().astype(np.float64), batch=host, dim=DIM, lens=list(host[1]))
    check_attention(c, turned.cpu().numpy(), y.view(m, HEADS, DIM), DIM ** -0.5)
    check_y(out, *oracle_y(layer.mats[3], y.cpu().numpy()), "last product")


def test_prompt_and_tokens():
    """Two prompts of different lengths in one ragged call, then tokens of
    both, one of them across a page's end."""
    rng = np.random.default_rng(3)
    layer, twin = Layer(rng, 8), L.KvCache.empty(8, KV, DIM)
    table = np.array([[5, 1, 2], [0, 7, 4]], np.int32)
    lens, start = np.array([70, 61], np.int32), np.array([0, 70, 131], np.int32)
    x = half(rng, 131, HIDDEN)
    batch = L.KvBatch(dev(lens), dev(table), 70, start=dev(start))
    check_block(layer, twin, layer.plan(dev(x)), x, np.concatenate([np.arange(70), np.arange(61)]).astype(np.int32),
                (start, lens, table, 2, 131, 70), batch)
    step = L.KvBatch(dev(lens), dev(table), 1)
    for t in range(6):
        lens += 1
        step.len.copy_(dev(lens))
        x = half(rng, 2, HIDDEN)
        check_block(layer, twin, layer.plan(dev(x)), x, lens - 1, (None, lens, table, 2, 2, 1), step)


def test_a_layer_captured_and_replayed_for_growing_lengths():
    """One graph of a token's whole block; each replay the next token, equal
    bitwise to the same tokens run eagerly on another cache."""
    rng = np.random.default_rng(5)
    layer = Layer(rng, 12)
    twin = L.KvCache.empty(12, KV, DIM)
    own = layer.cache
    table = dev(np.array([[3, 1, 4, 6, 9], [0, 7, 2, 5, 8]], np.int32))
    lens = dev(np.array([62, 100], np.int32))
    x = dev(half(rng, 2, HIDDEN))
    batch = L.KvBatch(lens, table, 1)
    plans = layer.plan(x)
    out = plans[2][4]
    ws = L.tern_kv_attention_workspace(own, batch, 2, HEADS)
    prompt = L.KvBatch(dev(np.array([62, 100], np.int32)), table, 100, start=dev(np.array([0, 62, 162], np.int32)))
    k, v = dev(half(rng, 162, KV, DIM)), dev(half(rng, 162, KV, DIM))
    for c in (own, twin):
        L.tern_kv_write(c, prompt, k, v)
    stream = torch.cuda.Stream()
    saved = [t.clone() for t in (own.k, own.v, own.k_scale, own.v_scale)]
    with torch.cuda.stream(stream):
        layer.run(plans, batch, stream.cuda_stream, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer.run(plans, batch, stream.cuda_stream, ws)
    for t, s in zip((own.k, own.v, own.k_scale, own.v_scale), saved):
        t.copy_(s)
    torch.cuda.synchronize()
    for t in range(70):
        x.copy_(dev(half(rng, 2, HIDDEN)))
        lens += 1
        torch.cuda.synchronize()
        layer.cache = twin
        layer.run(plans, batch)
        want = out.clone()
        out.fill_(-7)
        layer.cache = own
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"token {t}"
    for a, b in ((own.k, twin.k), (own.v, twin.v), (own.k_scale, twin.k_scale), (own.v_scale, twin.v_scale)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows,lens", [([1, 1, 1], [700, 3, 129]), ([20], [700]), ([150, 40], [400, 300]), ([600], [600])])
def test_attention_captured(rows, lens):
    rng = np.random.default_rng(rows[0])
    c = Case(rng, rows, lens, 2, 128)
    cache, batch = c.cache(), c.on_device()
    q = dev(half(rng, c.m, 4, 128))
    out = torch.empty_like(q)
    ws = L.tern_kv_attention_workspace(cache, batch, c.m, 4)

    def change(rep):
        q.copy_(dev(half(rng, c.m, 4, 128)))
        batch.len.copy_(dev(np.array([n - 5 * rep for n in lens], np.int32)))

    replay_checks(lambda s: L.tern_kv_attention(cache, batch, q, out=out, stream=s, ws=ws), change, [out])


def test_graphs_that_share_a_workspace():
    """Two captured calls of different shapes, replayed in turn."""
    rng = np.random.default_rng(11)
    cases = [Case(rng, [1], [3000], 2, 64), Case(rng, [3, 3], [900, 500], 2, 64)]
    held, ws = [], None
    for c in cases:
        cache, batch, q = c.cache(), c.on_device(), dev(half(rng, c.m, 4, 64))
        need = L.tern_kv_attention_workspace(cache, batch, c.m, 4)
        held.append((cache, batch, q, torch.empty_like(q), L.tern_kv_attention(cache, batch, q)))
        ws = need if ws is None or need.numel() > ws.numel() else ws
    stream, graphs = torch.cuda.Stream(), []
    for cache, batch, q, out, _ in held:
        with torch.cuda.stream(stream):
            L.tern_kv_attention(cache, batch, q, out=out, stream=stream.cuda_stream, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            L.tern_kv_attention(cache, batch, q, out=out, stream=stream.cuda_stream, ws=ws)
        graphs.append(g)
    for _ in range(3):
        for g, (_, _, _, out, want) in zip(graphs, held):
            out.fill_(9)
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_streams():
    """Calls on a stream of the caller's, with the workspaces and outputs that
    the binding makes: two at once on two streams."""
    rng = np.random.default_rng(13)
    c = Case(rng, [2, 2], [900, 700], 2, 128)
    cache, batch, q = c.cache(), c.on_device(), dev(half(rng, c.m, 8, 128))
    want = L.tern_kv_attention(cache, batch, q)
    freq, _ = K.frequencies(128, 1e4)
    rope, pos = L.Rope(dev(freq)), dev(np.arange(4, dtype=np.int32))
    turned = L.tern_rope(q, pos, rope)
    read = L.tern_kv_read(cache, batch)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        got = [(L.tern_kv_attention(cache, batch, q, stream=s.cuda_stream), L.tern_rope(q, pos, rope, stream=s.cuda_stream),
                *L.tern_kv_read(cache, batch, stream=s.cuda_stream)) for s in streams]
        torch.cuda.synchronize()
        for y, t, k, v in got:
            assert torch.equal(y, want) and torch.equal(t, turned) and torch.equal(k, read[0]) and torch.equal(v, read[1])


def test_threads_with_many_numbers_of_rows():
    """More than the descriptors that a batch keeps, from two threads."""
    rng = np.random.default_rng(15)
    c = Case(rng, [3, 5], [90, 70], 2, 64, ragged=True)
    cache, batch = c.cache(), c.on_device()
    want = [t[:8].clone() for t in L.tern_kv_read(cache, batch, rows=8)]
    torch.cuda.synchronize()
    bad = []

    def work(first):
        for rows in range(first, first + 150):
            if not all(torch.equal(a[:8], b) for a, b in zip(L.tern_kv_read(cache, batch, rows=rows), want)):
                bad.append(rows)

    threads = [threading.Thread(target=work, args=(first,)) for first in (8, 300)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_smaller_workspace_is_refused_and_bad_arguments():
    rng = np.random.default_rng(17)
    c = Case(rng, [1], [3000], 2, 64)
    cache, batch, q = c.cache(), c.on_device(), dev(half(rng, 1, 4, 64))
    with pytest.raises(L.TernError) as e:
        L.tern_kv_attention(cache, batch, q, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == L.TERN_E_WORKSPACE
    bad = [dict(q=q.float()), dict(q=q.cpu()), dict(q=q[0]), dict(q=q[:, :, :32]), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
           dict(q=q, out=torch.empty((1, 4, 64), device="cuda")), dict(q=q, ws=torch.empty(1 << 20, dtype=torch.uint8))]
    for kw in bad:
        with pytest.raises((ValueError, RuntimeError)):
            L.tern_kv_attention(cache, batch, **kw)
    for q_heads in (3, 5):
        with pytest.raises(L.TernError):
            L.tern_kv_attention(cache, batch, dev(half(rng, 1, q_heads, 64)))
    k = dev(half(rng, 1, 2, 64))
    freq, _ = K.frequencies(64, 1e4)
    rope = L.Rope(dev(freq), norm=dev(half(rng, 128)))
    for kw in (dict(k=k, v=k[:0]), dict(k=k, v=dev(half(rng, 1, 3, 64))), dict(k=k, v=k, rope=rope), dict(k=k, v=k, q=q),
               dict(k=k, v=k, q=dev(half(rng, 2, 4, 64)), q_rope=L.Rope(dev(freq)))):
        with pytest.raises(ValueError):
            L.tern_kv_write(cache, batch, **kw)
    with pytest.raises(ValueError):
        L.tern_kv_read(cache, batch, k=torch.empty((1, 2, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        L.tern_rope(k, dev(np.zeros(2, np.int32)), L.Rope(dev(freq)))
    with pytest.raises(ValueError):
        L.tern_rope(k, dev(np.zeros(1, np.int32)), L.Rope(dev(freq)), out=torch.empty((2, 2, 64), dtype=torch.float16, device="cuda"))
    with pytest.raises(L.TernError):
        L.KvCache.empty(2, 2, 96)

"""Cases of what stands between a decoder layer's products: rotary positions,
the writing and reading back of a cache held in 8 bits, and attention over it.

`run` computes a case either in its plain form (elementary torch operations)
or, with `own` set, through this package's entry points.  The cache is paged:
64 tokens a page, signed 8-bit codes, one FP32 scale for each (page, head) of
the keys and of the values; a value is code * scale.  Row j of a sequence's n
rows stands at position len - n + j, len counting the rows themselves.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64


# ---------------------------------------------------------------- cases
def _rope(name, m, heads, dim, rot, interleaved, base, scaling, first, norm):
    return dict(name=name, op="rope", m=m, heads=heads, dim=dim, rot=rot, interleaved=interleaved, base=base,
                scaling=scaling, first=first, norm=norm)


def _write(name, count, rows, most, ragged, heads, kv_heads, dim, rot, interleaved, scaling, norm, fused):
    return dict(name=name, op="write", count=count, rows=rows, most=most, ragged=ragged, heads=heads,
                kv_heads=kv_heads, dim=dim, rot=rot, interleaved=interleaved, base=1e6, scaling=scaling, norm=norm,
                fused=fused, empty=False)


def _read(name, count, rows, most, ragged, kv_heads, dim, out):
    return dict(name=name, op="read", count=count, rows=rows, most=most, ragged=ragged, kv_heads=kv_heads, dim=dim,
                empty=False, out=out)


def _attend(name, count, rows, most, ragged, heads, kv_heads, dim, window=0, causal=True, empty=False):
    return dict(name=name, op="attend", count=count, rows=rows, most=most, ragged=ragged, heads=heads,
                kv_heads=kv_heads, dim=dim, window=window, causal=causal, empty=empty)


def listed():
    return [
        # one token's queries and keys in an 8B-class layer, with the norm of each head: latency
        _rope("rope one token", 1, 40, 128, 128, False, 1e6, "none", 777, True),
        # a long prompt's chunk at far positions, half of each head turned in pairs, frequencies blended for a longer context
        _rope("rope far 5000", 5000, 32, 128, 64, True, 1e4, "ramp", 900000, False),
        # a decode batch of the 8B-class layer: a token each goes into pages that others began
        _write("write decode 48", 48, 1, 4000, True, 32, 8, 128, 128, False, "none", True, False),
        # a prefill chunk that begins inside a page, out of one fused projection
        _write("write prefill 4096", 1, 4096, 5001, False, 32, 8, 128, 128, False, "none", True, True),
        # prompts of many lengths, small heads that are not shared, positions scaled linearly
        _write("write ragged", 13, 300, 900, True, 12, 12, 64, 32, True, "linear", False, False),
        # a short prefix read back
        _read("read 77", 1, 77, 77, False, 8, 128, "f16"),
        # prefixes of many lengths read back
        _read("read prefixes", 6, 16000, 16000, True, 8, 128, "f32"),
        # one token after a medium context: latency
        _attend("attend one token", 1, 1, 4001, False, 32, 8, 128),
        # a decode batch with contexts of every length: the reading of the cache
        _attend("attend batch of 64", 64, 1, 8192, True, 32, 8, 128),
        # several tokens a sequence over long contexts (drafts to verify), one place of the batch empty
        _attend("attend drafts", 4, 5, 120000, True, 32, 8, 128, empty=True),
        # a prefill chunk after a thousand tokens
        _attend("attend prefill 2048", 1, 2048, 3048, False, 32, 8, 128),
        # prompts of many lengths, a sliding window, small heads that are not shared
        _attend("attend window ragged", 5, 1200, 1500, True, 12, 12, 64, window=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _shared(rng, dim):
    kv_heads = rng.choice((1, 2, 4, 8, 12))
    return kv_heads * rng.choice((1, 2, 3, 4, 5, 8) if kv_heads < 12 else (1, 2)), kv_heads


def draw(rng):
    op = rng.choice(("rope", "write", "read", "attend", "attend", "attend"))
    dim = rng.choice((64, 128, 128, 256))
    heads, kv_heads = _shared(rng, dim)
    rot = dim if rng.random() < 0.5 else 2 * rng.randint(1, dim // 2)
    scaling = rng.choice(("none", "linear", "ramp"))
    if op == "rope":
        m = _log(rng, 1, max(2, 5000 * 32 * 128 // (heads * dim)))
        c = _rope("", min(m, 20000), heads, dim, rot, rng.random() < 0.5, rng.choice((1e4, 1e6)), scaling,
                  _log(rng, 1, 1000000), rng.random() < 0.5)
    elif op == "write":
        rows = 1 if rng.random() < 0.4 else min(_log(rng, 2, 4096), 25000000 // ((heads + 3 * kv_heads) * dim))
        count = _log(rng, 1, max(1, min(64, 25000000 // (rows * (heads + 3 * kv_heads) * dim))))
        c = _write("", count, rows, rows + _log(rng, 1, 1000), rng.random() < 0.6, heads, kv_heads, dim, rot,
                   rng.random() < 0.5, scaling, rng.random() < 0.5, rng.random() < 0.5)
    elif op == "read":
        rows = _log(rng, 1, 16000)
        count = _log(rng, 1, max(1, min(64, 3 * 16000 * 1024 // (rows * kv_heads * dim))))
        c = _read("", count, rows, rows + _log(rng, 1, 500), rng.random() < 0.6, kv_heads, dim, rng.choice(("f16", "f32")))
    else:
        rows = 1 if rng.random() < 0.5 else _log(rng, 2, 16) if rng.random() < 0.5 else _log(rng, 17, 2048)
        rows = min(rows, 2048 * 32 * 128 // (heads * dim))
        most = min(rows + _log(rng, 1, 100000 if rows < 17 else 1000), 64 * 4000 * 1024 // (kv_heads * dim))
        pairs = 2048 * 2000 * 32 * 128 // (rows * most * heads * dim)
        count = _log(rng, 1, max(1, min(64, 64 * 4000 * 1024 // (most * kv_heads * dim), pairs)))
        causal = rng.random() < 0.85
        c = _attend("", count, rows, most, rng.random() < 0.7, heads, kv_heads, dim,
                    _log(rng, 8, 2000) if causal and rng.random() < 0.3 else 0, causal, count > 1 and rng.random() < 0.3)
    del c["name"]
    return c


def _lengths(case):
    """The sequences' rows and lengths, by the case alone."""
    rng = random.Random(case["count"] * 1000003 + case["rows"] * 1009 + case["most"])
    rows, lens = [], []
    for i in range(case["count"]):
        if not case["ragged"] or i == case["count"] // 2:
            n, total = case["rows"], case["most"]
        else:
            n = case["rows"] if case["rows"] < 17 else rng.randint(1, case["rows"])
            total = n + int((case["most"] - case["rows"]) * rng.random())
        if case["empty"] and i == case["count"] - 1:
            total = 0  # its rows stand before the sequence's beginning
        rows.append(n)
        lens.append(total)
    return rows, lens


# ---------------------------------------------------------------- inputs
def _frequencies(case):
    """Radians a token, FP64 [rot / 2]: base^(-2i/rot), divided by 4, or
    blended with that between the pairs that turn 32 times and once in 4096
    tokens."""
    rot = case["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    f = case["base"] ** (-2 * i / rot)
    if case["scaling"] == "linear":
        return f / 4
    if case["scaling"] == "ramp":
        at = [0.5 * rot * math.log(4096 / (turns * 2 * math.pi)) / math.log(case["base"]) for turns in (32, 1)]
        low, high = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        keep = 1 - ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        return f * keep + f / 4 * (1 - keep)
    return f


def _codes(gen, pages, heads, dim, keys):
    """Codes as the cache holds them, bytes code + 128 [pages][heads][64 * dim]
    in the order of its pages, bell-shaped, for the keys with a few channels
    that are four times as large, and scales of 8 significant bits."""
    if keys:  # token 16a + 4t + i, dimension 64c + 16r + b: [c][t][r][a][i][b]
        order = (dim // 64, 4, 4, 4, 4, 16)
        loud = torch.rand((heads, dim), generator=gen, device="cuda") < 0.05
        spread = torch.where(loud, 48.0, 12.0).view(heads, dim // 64, 1, 4, 1, 1, 16)
    else:  # token 16a + j, dimension 16c + e: [c][a][e][j]
        order, spread = (dim // 16, 4, 16, 16), 30.0
    codes = torch.empty((pages, heads, *order), dtype=torch.uint8, device="cuda")
    some = max(1, (1 << 27) // (heads * PAGE * dim))
    for p in range(0, pages, some):
        x = torch.randn(codes[p:p + some].shape, generator=gen, device="cuda") * spread
        codes[p:p + some] = x.round_().clamp_(-127, 127).add_(128).to(torch.uint8)
    scale = torch.randint(128, 256, (pages, heads), generator=gen, device="cuda").float() * 2.0 ** (-11 if keys else -12)
    return codes.view(pages, heads, PAGE, dim), scale


def _natural(codes, keys):
    """Such codes as int8 [pages][heads][64][dim] in the order of tokens and
    dimensions, as a program without this package would keep them."""
    p, h, _, d = codes.shape
    if keys:
        v = codes.view(p, h, d // 64, 4, 4, 4, 4, 16).permute(0, 1, 5, 3, 6, 2, 4, 7)
    else:
        v = codes.view(p, h, d // 16, 4, 16, 16).permute(0, 1, 3, 5, 2, 4)
    return (v.contiguous() ^ 128).view(torch.int8).view(p, h, PAGE, d)


def _tensor(v, kind=torch.int32):
    return torch.tensor(v, dtype=kind, device="cuda")


def _places(rows, lens, table):
    """Of every row: its sequence, its position, and the page it lies in."""
    n, total = _tensor(rows, torch.int64), _tensor(lens, torch.int64)
    seq = torch.repeat_interleave(torch.arange(len(rows), device="cuda"), n)
    first = n.cumsum(0) - n
    pos = total[seq] - n[seq] + torch.arange(seq.numel(), device="cuda") - first[seq]
    return seq, pos, table[seq, pos.clamp(min=0) // PAGE].long()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dim = case["dim"]
    if own:
        from ternary_weight_only_tern_amd import lib as L
        s["lib"] = L
    if "rot" in case:
        s["freq"], s["amp"] = _frequencies(case), 1.0 if case["scaling"] != "ramp" else 0.1 * math.log(4) + 1
        norms = [(1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")).half() if case["norm"] else None for _ in range(2)]
        s["q_norm"], s["k_norm"] = norms
    if case["op"] == "rope":
        m = case["m"]
        s["x"] = torch.randn((m, case["heads"], dim), generator=gen, device="cuda").half()
        s["pos"] = case["first"] + torch.arange(m, dtype=torch.int32, device="cuda")
        if own:
            s["rope"] = L.Rope(s["freq"], case["interleaved"], s["amp"], s["q_norm"], 1e-6)
            s["y"] = torch.empty_like(s["x"])
        return s

    heads = case["kv_heads"]
    rows, lens = _lengths(case)
    m = sum(rows)
    need = [-(-t // PAGE) for t in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32).tolist()
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (max(need) - n))
        at += n
    s["table"] = _tensor(table)
    s["len"] = _tensor(lens)
    s["seq"], s["pos"], s["at"] = _places(rows, lens, s["table"])
    k, ks = _codes(gen, pages, heads, dim, True)
    v, vs = _codes(gen, pages, heads, dim, False)
    if case["op"] == "write":  # tokens before these were smaller, some of them
        ks, vs = (f * 2.0 ** -torch.randint(0, 4, f.shape, generator=gen, device="cuda") for f in (ks, vs))
    if case["op"] == "attend":
        s["q"] = torch.randn((m, case["heads"], dim), generator=gen, device="cuda").half()
        s["j"] = s["pos"] - s["len"].long()[s["seq"]] + _tensor(rows, torch.int64)[s["seq"]]
        s["scale"] = dim ** -0.5
    if case["op"] == "write":
        n, width = (case["heads"] + 2 * heads) * dim, [case["heads"] * dim, heads * dim, heads * dim]
        row = torch.randn((m, n), generator=gen, device="cuda")
        row *= torch.exp(0.3 * torch.randn((m, 1), generator=gen, device="cuda"))
        if case["fused"]:
            parts = row.half().split(width, dim=1)
        else:
            parts = [t.half().contiguous() for t in row.split(width, dim=1)]
        s["q"], s["k"], s["v"] = (t.unflatten(1, (-1, dim)) for t in parts)
        # the pages that the rows lie in, and every token of a sequence from its first such page on
        s["met"], s["row_met"] = torch.unique(s["at"], return_inverse=True)
        first = [(t - r) // PAGE * PAGE for t, r in zip(lens, rows)]
        back = [t - f for t, f in zip(lens, first)]
        s["back"] = _places(back, lens, s["table"])
    if not own:
        s["kc"], s["ks"], s["vc"], s["vs"] = _natural(k, True), ks, _natural(v, False), vs
    if own:
        s["cache"] = L.KvCache(k, v, ks, vs)
        starts = lambda n: None if len(set(n)) == 1 else _tensor([sum(n[:i]) for i in range(len(n) + 1)])
        batch = lambda n: L.KvBatch(s["len"], s["table"], max(n), start=starts(n), max_len=max(lens))
        s["batch"] = batch(rows)
        if case["op"] == "attend":
            s["y"] = torch.empty((m, case["heads"], dim), dtype=torch.float16, device="cuda")
            s["ws"] = L.tern_kv_attention_workspace(s["cache"], s["batch"], m, case["heads"])
        else:
            if case["op"] == "write":
                s["rope"], s["k_rope"] = (L.Rope(s["freq"], case["interleaved"], s["amp"], t, 1e-6) for t in norms)
                s["q_out"] = torch.empty((m, case["heads"], dim), dtype=torch.float16, device="cuda")
                s["batch_back"], m = batch(back), sum(back)
            kind = torch.float32 if case.get("out") == "f32" else torch.float16
            s["k_out"], s["v_out"] = (torch.empty((m, heads, dim), dtype=kind, device="cuda") for _ in range(2))
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _call(s)
    if s["op"] == "rope":
        return _plain_rope(s, s["x"], s["pos"], s["q_norm"])
    if s["op"] == "write":
        return _plain_write(s)
    if s["op"] == "read":
        return _plain_read(s, s["pos"], s["at"])
    return _plain_attend(s)


def _call(s):
    L = s["lib"]
    if s["op"] == "rope":
        return L.tern_rope(s["x"], s["pos"], s["rope"], out=s["y"])
    if s["op"] == "write":
        L.tern_kv_write(s["cache"], s["batch"], s["k"], s["v"], rope=s["k_rope"], q=s["q"], q_rope=s["rope"], q_out=s["q_out"])
        return s["q_out"], *L.tern_kv_read(s["cache"], s["batch_back"], k=s["k_out"], v=s["v_out"])
    if s["op"] == "read":
        return L.tern_kv_read(s["cache"], s["batch"], k=s["k_out"], v=s["v_out"])
    return L.tern_kv_attention(s["cache"], s["batch"], s["q"], scale=s["scale"], window=s["window"], causal=s["causal"],
                               out=s["y"], ws=s["ws"])


def _plain_rope(s, x, pos, norm):
    y = x.float()
    if norm is not None:
        y = y / torch.sqrt((y * y).mean(dim=-1, keepdim=True) + 1e-6) * norm.float()
    angle = pos.double().unsqueeze(1) * s["freq"]
    c, d = ((s["amp"] * t).float().unsqueeze(1) for t in (torch.cos(angle), torch.sin(angle)))
    rot = s["rot"]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if s["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:rot])
    a, b = a * c - b * d, b * c + a * d
    turned = torch.stack((a, b), dim=-1).flatten(-2) if s["interleaved"] else torch.cat((a, b), dim=-1)
    return torch.cat((turned, y[..., rot:]), dim=-1).to(torch.float16)


def _plain_quantise(s, codes, scale, x):
    """The rows of x into their pages.  A page whose first token is among them,
    or that holds nothing but zeros, takes its largest value / 127, rounded up
    to 8 significant bits; another doubles its scale until they fit."""
    most = x.float().abs().amax(dim=-1)
    met, row = s["met"], s["row_met"]
    top = torch.zeros((met.numel(), most.shape[1]), device=x.device).index_reduce_(0, row, most, "amax")
    new = torch.zeros(met.numel(), dtype=torch.bool, device=x.device)
    new[row[s["pos"] % PAGE == 0]] = True
    need = (((top / 127).view(torch.int32) + 0xFFFF) & -65536).view(torch.float32)
    old = scale[met]
    base = torch.where(new.unsqueeze(1) | (old == 0), need, old)
    part, power = torch.frexp(torch.where(base > 0, top / (127 * base), 0))
    power = (power - (part == 0.5).int()).clamp(min=0)
    scale[met] = torch.ldexp(base, power)
    shrink = torch.ldexp(torch.ones_like(base), -power)
    codes[met] = torch.round(codes[met].float() * shrink[..., None, None]).to(torch.int8)
    by = scale[s["at"]].unsqueeze(-1)
    code = torch.where(by > 0, torch.round(x.float() / by), 0)
    codes[s["at"], :, s["pos"] % PAGE] = code.to(torch.int8)


def _plain_write(s):
    q = _plain_rope(s, s["q"], s["pos"], s["q_norm"])
    _plain_quantise(s, s["kc"], s["ks"], _plain_rope(s, s["k"], s["pos"], s["k_norm"]))
    _plain_quantise(s, s["vc"], s["vs"], s["v"])
    return q, *_plain_read(s, s["back"][1], s["back"][2])


def _plain_read(s, pos, at):
    kind = torch.float32 if s.get("out") == "f32" else torch.float16
    return tuple((s[c][at, :, pos % PAGE].float() * s[f][at].unsqueeze(-1)).to(kind) for c, f in (("kc", "ks"), ("vc", "vs")))


def _plain_attend(s):
    q, table = s["q"], s["table"].long()
    count, most = table.shape
    heads, dim = s["kv_heads"], s["dim"]
    group, rows = s["heads"] // heads, s["rows"]
    k, v = ((s[c][table.clamp(min=0)].float() * s[f][table.clamp(min=0)][..., None, None]).transpose(1, 2).reshape(count * heads, most * PAGE, dim)
            for c, f in (("kc", "ks"), ("vc", "vs")))
    batch = torch.zeros((count, rows, heads, group, dim), device=q.device)
    batch[s["seq"], s["j"]] = q.float().unflatten(1, (heads, group))
    batch = batch.permute(0, 2, 1, 3, 4).reshape(count * heads, rows * group, dim)
    pos = torch.full((count, rows), -1, dtype=torch.int64, device=q.device)
    pos[s["seq"], s["j"]] = s["pos"]
    token = torch.arange(most * PAGE, device=q.device)
    pos = pos.unsqueeze(2)
    sees = (token < s["len"].long()[:, None, None]) & (pos >= 0)
    if s["causal"]:
        sees = sees & (token <= pos)
    if s["window"]:
        sees = sees & (token > pos - s["window"])
    sees = sees[:, None, :, None, :].expand(count, heads, rows, group, -1).reshape(count * heads, rows * group, -1)
    score = torch.bmm(batch, k.transpose(1, 2).contiguous()).mul_(s["scale"]).masked_fill_(~sees, -math.inf)
    top = score.amax(dim=-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    y = torch.bmm(p, v) / torch.where(total > 0, total, 1.0)
    y = y.view(count, heads, rows, group, dim).transpose(1, 2).reshape(count, rows, heads * group, dim)[s["seq"], s["j"]]
    return y.to(torch.float16)


# ---------------------------------------------------------------- what a pass cannot do without
def _seen(case, n, total):
    """(pairs of rows and tokens, tokens that some row sees) of one sequence."""
    if total < n:
        return 0, 0
    if not case["causal"]:
        return n * total, total
    last = np.arange(total - n + 1, total + 1, dtype=np.int64)
    if case["window"]:
        return int(np.minimum(last, case["window"]).sum()), min(total, case["window"] + n - 1)
    return int(last.sum()), total


def work(case):
    dim = case["dim"]
    if case["op"] == "rope":
        values = case["m"] * case["heads"] * dim
        return {"bytes": 4 * values + 4 * case["m"], "flops": 6 * values}
    heads = case["kv_heads"]
    rows, lens = _lengths(case)
    m = sum(rows)
    if case["op"] == "read":
        return {"bytes": 2 * m * heads * dim * (5 if case["out"] == "f32" else 3) + 8 * heads * m // PAGE, "flops": 2 * m * heads * dim}
    if case["op"] == "write":
        back = sum(t - (t - r) // PAGE * PAGE for t, r in zip(lens, rows))
        values = m * heads * dim
        return {"bytes": 4 * m * case["heads"] * dim + 2 * values * 3 + 2 * back * heads * dim * 3,
                "flops": 6 * m * case["heads"] * dim + 12 * values + 2 * back * heads * dim}
    pairs, tokens = (sum(v) for v in zip(*(_seen(case, n, t) for n, t in zip(rows, lens))))
    return {"bytes": 2 * tokens * heads * dim + 8 * heads * tokens // PAGE + 4 * m * case["heads"] * dim,
            "flops": 4 * pairs * case["heads"] * dim}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        return _exact_rope(s, s["x"], s["pos"], s["q_norm"])
    if case["op"] == "read":
        return _exact_read(s, s["pos"], s["at"])
    if case["op"] == "write":
        k = _exact_rope(s, s["k"], s["pos"], s["k_norm"]).half()  # what the cache is given has 16 bits
        _exact_quantise(s, "kc", "ks", k.double())
        _exact_quantise(s, "vc", "vs", s["v"].double())
        return _exact_rope(s, s["q"], s["pos"], s["q_norm"]), *_exact_read(s, s["back"][1], s["back"][2])
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    heads, dim = s["kv_heads"], s["dim"]
    group = s["heads"] // heads
    for i in range(case["count"]):
        mine = (s["seq"] == i).nonzero().flatten()
        total = int(s["len"][i])
        pos = s["pos"][mine]
        if not total or not mine.numel():
            continue
        token = torch.arange(total, device="cuda")
        page, place = s["table"][i].long()[token // PAGE], token % PAGE
        for h in range(heads):
            k = s["kc"][page, h, place].double() * s["ks"][page, h].double().unsqueeze(1)
            v = s["vc"][page, h, place].double() * s["vs"][page, h].double().unsqueeze(1)
            dark = pos.unsqueeze(1) < 0
            if case["causal"]:
                dark = dark | (token > pos.unsqueeze(1))
            if case["window"]:
                dark = dark | (token <= pos.unsqueeze(1) - case["window"])
            for g in range(h * group, h * group + group):
                z = (s["q"][mine, g].double() @ k.t()) * s["scale"]
                w = torch.softmax(z.masked_fill(dark, -math.inf), dim=1)
                y[mine, g] = w.nan_to_num(nan=0.0) @ v
    return y


def _exact_rope(s, x, pos, norm):
    """Pair by pair as complex numbers."""
    x = x.double()
    if norm is not None:
        x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * norm.double()
    rot = s["rot"]
    half = rot // 2
    even = torch.arange(half, device=x.device) * (2 if s["interleaved"] else 1)
    odd = even + (1 if s["interleaved"] else half)
    turn = torch.polar(torch.full((pos.numel(), 1, half), float(s["amp"]), dtype=torch.float64, device=x.device),
                       torch.outer(pos.double(), s["freq"]).unsqueeze(1))
    z = torch.complex(x[..., even], x[..., odd]) * turn
    y = x.clone()
    y[..., even], y[..., odd] = z.real, z.imag
    return y


def _exact_quantise(s, name, factor, x):
    """Page by page."""
    pos = s["pos"]
    where = s["at"].tolist()
    order = {}
    for r, p in enumerate(where):
        order.setdefault(p, []).append(r)
    host = pos.tolist()
    for p, r in order.items():
        new = x[r]
        top = new.abs().amax(dim=(0, 2)).cpu().numpy()
        old = s[factor][p].double().cpu().numpy()
        fraction, power = np.frexp(top / 127)
        least = np.ldexp(np.ceil(fraction * 256), power - 8)
        fresh = (old == 0) | any(host[i] % PAGE == 0 for i in r)
        start = np.where(fresh, least, old)
        while (low := top > 127 * start).any():
            start = np.where(low, 2 * start, start)
        ratio = torch.from_numpy(np.where(fresh, 1.0, old / np.where(start > 0, start, 1.0))).cuda()
        s[name][p] = torch.round(s[name][p].double() * ratio[:, None, None]).to(torch.int8)
        by = torch.from_numpy(start).cuda()
        s[factor][p] = by.float()
        code = torch.round(new / torch.where(by > 0, by, 1.0)[None, :, None])
        s[name][p][:, pos[r] % PAGE] = code.to(torch.int8).transpose(0, 1)


def _exact_read(s, pos, at):
    return tuple(s[c][at, :, pos % PAGE].double() * s[f][at].double().unsqueeze(-1) for c, f in (("kc", "ks"), ("vc", "vs")))

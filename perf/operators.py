"""Cases of the 4-bit linear layers: the product with 4-bit weights and group
scales, the routing of tokens to experts, and the routed experts' products.

`run` computes a case either in its plain form (elementary torch operations)
or, with `own` set, through this package's entry points.  4-bit weights are
codes q in 0..15 with an FP16 scale and optionally an integer zero point (8
without one) per group:
W[n][k] = scale[n][k // group] * (q[n][k] - zero[n][k // group]).
Eight consecutive codes of a row fill a little-endian 32-bit word, the one at
offset o in bits 16 * (o % 2) + 4 * (o // 2) and up, as the 2-bit trits' words
are filled: its bytes hold the offsets (0, 2), (4, 6), (1, 3), (5, 7).
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases
def _q4(name, m, n, k, group, zero, out):
    return dict(name=name, op="q4", m=m, n=n, k=k, group=group, zero=zero, out=out)


def _route(name, m, experts, topk, score, bias, groups, best, keep, renorm, scale, logits, masked):
    return dict(name=name, op="route", m=m, experts=experts, topk=topk, score=score, bias=bias, groups=groups,
                best=best, keep=keep, renorm=renorm, scale=scale, logits=logits, masked=masked)


def _experts(name, m, experts, topk, hidden, inner, group, zero, skipped):
    return dict(name=name, op="experts", m=m, experts=experts, topk=topk, hidden=hidden, inner=inner, group=group,
                zero=zero, skipped=skipped)


def listed():
    return [
        # one token through a square projection of the 8B-class layer: latency
        _q4("q4 token 4096x4096", 1, 4096, 4096, 128, False, "f16"),
        # one token through a vocabulary head, kept at 4 bits beside ternary layers: a long read
        _q4("q4 token head", 1, 131072, 2560, 128, True, "f16"),
        # a ragged decode batch through the 8B-class gate/up projection, FP32 outputs
        _q4("q4 batch of 13", 13, 12288, 4096, 64, True, "f32"),
        # a short prompt through the 4B-class down projection, the smallest groups
        _q4("q4 prompt of 77", 77, 2560, 9728, 32, False, "f16"),
        # a prefill chunk through the 8B-class gate/up projection
        _q4("q4 prefill 512", 512, 12288, 4096, 128, False, "f16"),
        # one token's routing: softmax, renormalised
        _route("route one token", 1, 64, 8, "softmax", False, 1, 1, 1, True, 1.0, "f16", False),
        # a decode batch: sigmoid scores, a balance bias, groups judged by their two best
        _route("route batch of 37", 37, 256, 8, "sigmoid", True, 8, 2, 4, True, 2.5, "f32", False),
        # a long prefill with the same router
        _route("route prefill 16384", 16384, 256, 8, "sigmoid", True, 8, 2, 4, True, 2.5, "f32", False),
        # padded tokens and disabled experts (logits of minus infinity), odd sizes, plain softmax weights
        _route("route masked 5001", 5001, 100, 6, "softmax", False, 1, 1, 1, False, 1.0, "f16", True),
        # one token through its experts: latency and the reading of eight experts' weights
        _experts("experts one token", 1, 64, 8, 2560, 1024, 128, False, False),
        # an odd batch, small groups, zero points, slots that name no expert
        _experts("experts batch of 21", 21, 16, 2, 4096, 1056, 32, True, True),
        # a prefill chunk: every expert has some hundred tokens
        _experts("experts prefill 2048", 2048, 64, 8, 2560, 1024, 128, False, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("q4", "q4", "route", "experts"))
    if op == "q4":
        group = rng.choice((32, 64, 128))
        m = 1 if rng.random() < 0.3 else _log(rng, 1, 512)
        k = group * max(1, _log(rng, 64, 12288) // group)
        n = max(1, min(_log(rng, 64, 32768), 512 * 12288 * 4096 // (m * k)))
        c = _q4("", m, n, k, group, rng.random() < 0.5, rng.choice(("f16", "f32")))
    elif op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        size = rng.randint(2, 256 // groups)
        experts = groups * size
        keep = rng.randint(1, groups)
        topk = rng.randint(1, min(16, keep * size))
        bias = rng.random() < 0.6
        best = rng.randint(1, 2)
        c = _route("", _log(rng, 1, 16384), experts, topk, rng.choice(("softmax", "sigmoid")), bias, groups, best, keep,
                   rng.random() < 0.6, rng.choice((1.0, 2.5)), rng.choice(("f16", "f32")), rng.random() < 0.3)
    else:
        group = rng.choice((32, 64, 128))
        experts = rng.choice((4, 8, 16, 32, 60, 64))
        topk = rng.randint(1, min(8, experts))
        hidden = group * max(1, _log(rng, 256, 2560) // group)
        inner = group * max(1, _log(rng, 128, 1024) // group)
        c = _experts("", _log(rng, 1, 2048), experts, topk, hidden, inner, group, rng.random() < 0.5,
                     rng.random() < 0.3)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs
def _weights(gen, lead, n, k, group, zero):
    """Codes, scales and zero points as a 4-bit quantizer leaves them: codes
    bell-shaped around the zero point, scales within a factor of a few."""
    z = None
    mid = 8
    if zero:
        z = torch.randint(5, 12, (*lead, n, k // group), generator=gen, device="cuda", dtype=torch.uint8)
        mid = z.to(torch.float16).repeat_interleave(group, dim=-1)
    q = torch.empty((*lead, n, k), dtype=torch.float16, device="cuda").normal_(0.0, 2.7, generator=gen)
    q = (q + mid).round_().clamp_(0, 15).to(torch.uint8)
    codes = torch.stack([q[..., o::8] | (q[..., o + 2::8] << 4) for o in (0, 4, 1, 5)], dim=-1).flatten(-2)
    scale = torch.empty((*lead, n, k // group), dtype=torch.float32, device="cuda").uniform_(0.002, 0.012, generator=gen)
    return codes.contiguous(), scale.to(torch.float16), z


def _activations(gen, m, k):
    """FP16, unit normal with a few channels that are eight times as large."""
    x = torch.randn((m, k), generator=gen, device="cuda")
    loud = torch.rand((1, k), generator=gen, device="cuda") < 0.01
    return torch.where(loud, 8 * x, x).to(torch.float16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    m = case["m"]
    if case["op"] == "q4":
        s["w"] = _weights(gen, (), case["n"], case["k"], case["group"], case["zero"])
        s["x"] = _activations(gen, m, case["k"])
    elif case["op"] == "route":
        e = case["experts"]
        logits = 1.5 * torch.randn((m, e), generator=gen, device="cuda")
        if case["masked"]:
            off = torch.rand((m, e), generator=gen, device="cuda") < 0.2
            off[6::97] = True
            logits = logits.masked_fill(off, -math.inf)
        s["l"] = logits.to(torch.float16 if case["logits"] == "f16" else torch.float32)
        s["b"] = 0.1 * torch.randn((e,), generator=gen, device="cuda") if case["bias"] else None
    else:
        e, h, i = case["experts"], case["hidden"], case["inner"]
        s["gate_up"] = _weights(gen, (e,), 2 * i, h, case["group"], case["zero"])
        s["down"] = _weights(gen, (e,), h, i, case["group"], case["zero"])
        s["x"] = _activations(gen, m, h)
        liked = torch.randn((m, e), generator=gen, device="cuda") + 0.5 * torch.randn((1, e), generator=gen, device="cuda")
        top = torch.topk(liked, case["topk"], dim=1)
        s["ids"] = top.indices.to(torch.int32).contiguous()
        s["g"] = torch.softmax(top.values, dim=1).contiguous()
        if case["skipped"]:
            s["ids"].masked_fill_(torch.rand(s["ids"].shape, generator=gen, device="cuda") < 0.2, -1)
    if own:  # the handles, outputs and workspaces that a program keeps between calls
        from ternary_weight_only_tern_amd import lib as L
        s["lib"] = L
        if case["op"] == "q4":
            f32 = case["out"] == "f32"
            s["handle"] = L.Q4Matrix(*s["w"])
            s["y_dtype"] = L.TERN_F32 if f32 else L.TERN_F16
            s["y"] = torch.empty((m, case["n"]), dtype=torch.float32 if f32 else torch.float16, device="cuda")
            s["ws"] = L.tern_q4_workspace(s["handle"], m)
        elif case["op"] == "route":
            s["score_kind"] = L.TERN_SCORE_SIGMOID if case["score"] == "sigmoid" else L.TERN_SCORE_SOFTMAX
            s["ids"] = torch.empty((m, case["topk"]), dtype=torch.int32, device="cuda")
            s["g"] = torch.empty((m, case["topk"]), dtype=torch.float32, device="cuda")
        else:
            s["handles"] = L.Q4Matrix(*s["gate_up"]), L.Q4Matrix(*s["down"])
            s["y"] = torch.empty((m, case["hidden"]), dtype=torch.float16, device="cuda")
            s["ws"] = L.tern_q4_experts_workspace(*s["handles"], m, case["topk"])
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _call(s)
    if s["op"] == "q4":
        y = s["x"].float() @ _dense(*s["w"]).t()
        return y if s["out"] == "f32" else y.to(torch.float16)
    if s["op"] == "route":
        return _plain_route(s)
    return _plain_experts(s)


def _call(s):
    L = s["lib"]
    if s["op"] == "q4":
        return L.tern_q4_gemm(s["handle"], s["x"], s["y_dtype"], out=s["y"], ws=s["ws"])
    if s["op"] == "route":
        return L.tern_route(s["l"], s["topk"], score=s["score_kind"], bias=s["b"], groups=s["groups"],
                            group_best=s["best"], keep_groups=s["keep"], renorm=s["renorm"], scale=s["scale"],
                            ids=s["ids"], weights=s["g"])
    return L.tern_q4_experts(*s["handles"], s["x"], s["ids"], s["g"], out=s["y"], ws=s["ws"])


def _dense(codes, scale, zero):
    """The weights in FP32."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1)  # in a word: offsets 0 2 4 6, then 1 3 5 7
    q = q.reshape(*codes.shape[:-1], -1, 2, 4).transpose(-1, -2)
    q = q.reshape(*scale.shape, -1).float()
    q = q - (8.0 if zero is None else zero.float().unsqueeze(-1))
    return (q * scale.float().unsqueeze(-1)).flatten(-2)


def _plain_route(s):
    """Scores and selection in 64 bits: whole numbers hang on their order.
    NaN counts as minus infinity and plus infinity as FP32's largest value;
    an expert whose key is minus infinity is not chosen (id -1, weight 0)."""
    least = -math.inf
    l = s["l"].double().nan_to_num(nan=least, posinf=torch.finfo(torch.float32).max, neginf=least)
    m, e = l.shape
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-l))
    else:
        score = torch.exp(l - l.max(dim=1, keepdim=True).values.clamp(min=-3e38))
        score = score / score.sum(dim=1, keepdim=True).clamp(min=1)
    if s["b"] is None and (s["groups"] == 1 or s["best"] == 1):
        key = l  # both scores grow with the logit
    else:
        key = score if s["b"] is None else score + s["b"].double()
        key = torch.where(l == least, least, key).nan_to_num(nan=least, posinf=math.inf, neginf=least)
    if s["groups"] > 1:
        per = key.view(m, s["groups"], -1).sort(dim=2, descending=True).values[:, :, :s["best"]]
        total = torch.where(per == least, 0.0, per).sum(dim=2)
        total = torch.where(per[:, :, 0] == least, least, total)
        order = total.sort(dim=1, descending=True, stable=True).indices
        kept = torch.zeros_like(total, dtype=torch.bool).scatter_(1, order[:, :s["keep"]], True)
        key = torch.where(kept.repeat_interleave(e // s["groups"], dim=1), key, least)
    top = key.sort(dim=1, descending=True, stable=True)
    chosen, ids = top.values[:, :s["topk"]] > least, top.indices[:, :s["topk"]]
    g = torch.where(chosen, score.gather(1, ids), 0.0)
    if s["renorm"]:
        total = g.sum(dim=1, keepdim=True)
        g = torch.where(total > 0, g / total, 0.0)
    return torch.where(chosen, ids, -1).to(torch.int32), (g * s["scale"]).float()


def _swiglu(gu):
    gate, up = gu.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _plain_experts(s):
    """Few tokens: each slot with its own expert's weights.  Many: the slots
    sorted by expert, one padded batch of products over all experts."""
    x, ids, g = s["x"].float(), s["ids"].long(), s["g"]
    m, topk = ids.shape
    experts = s["experts"]
    if m * topk <= experts:
        pick = ids.clamp(min=0).flatten()
        row = x.repeat_interleave(topk, dim=0).unsqueeze(-1)
        h = _swiglu(torch.bmm(_dense(*_of(s["gate_up"], pick)), row).squeeze(-1))
        y = torch.bmm(_dense(*_of(s["down"], pick)), h.unsqueeze(-1)).view(m, topk, -1)
    else:
        flat = torch.where(ids < 0, experts, ids).flatten()
        order = flat.sort(stable=True).indices
        count = torch.bincount(flat, minlength=experts + 1)
        place = torch.empty_like(flat)
        place[order] = torch.arange(flat.numel(), device=flat.device) - (count.cumsum(0) - count)[flat[order]]
        most = max(1, int(count[:experts].max()))
        at = torch.where(flat < experts, flat * most + place, experts * most)
        rows = torch.zeros((experts * most + 1, x.shape[1]), device=x.device)
        rows[at] = x.repeat_interleave(topk, dim=0)
        rows = rows[:-1].view(experts, most, -1).transpose(1, 2).contiguous()
        h = _swiglu(torch.bmm(_dense(*s["gate_up"]), rows).transpose(1, 2))
        out = torch.bmm(_dense(*s["down"]), h.transpose(1, 2).contiguous()).transpose(1, 2)
        out = torch.cat((out.reshape(experts * most, -1), torch.zeros((1, out.shape[2]), device=x.device)))
        y = out[at].view(m, topk, -1)
    y = torch.where((ids < 0).unsqueeze(-1), 0.0, y * g.unsqueeze(-1))
    return y.sum(dim=1).to(torch.float16)


def _of(w, pick):
    return [None if t is None else t[pick] for t in w]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    m = case["m"]
    if case["op"] == "q4":
        n, k = case["n"], case["k"]
        w = n * k // 2 + n * (k // case["group"]) * (3 if case["zero"] else 2)
        return {"bytes": w + 2 * m * k + m * n * (4 if case["out"] == "f32" else 2), "flops": 2 * m * n * k}
    if case["op"] == "route":
        e = case["experts"]
        return {"bytes": m * e * (2 if case["logits"] == "f16" else 4) + 8 * m * case["topk"] + (4 * e if case["bias"] else 0),
                "flops": 4 * m * e}
    h, i, e, topk = case["hidden"], case["inner"], case["experts"], case["topk"]
    slots = m * topk * (0.8 if case["skipped"] else 1)
    met = e * (1 - (1 - slots / (m * e)) ** m)
    per = 3 * h * i * (0.5 + (3 if case["zero"] else 2) / case["group"])
    return {"bytes": met * per + 4 * m * h + 8 * m * topk, "flops": 6 * slots * h * i}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "q4":
        return _exact_rows(s["x"].double(), *s["w"])
    if case["op"] == "route":
        return _exact_route(s)
    x, g = s["x"].double(), s["g"].double()
    y = torch.zeros((case["m"], case["hidden"]), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        t, slot = (s["ids"] == e).nonzero(as_tuple=True)
        if t.numel():
            gu = _exact_rows(x[t], *_of(s["gate_up"], e))
            i = case["inner"]
            h = torch.sigmoid(gu[:, :i]) * gu[:, :i] * gu[:, i:]
            y.index_add_(0, t, _exact_rows(h, *_of(s["down"], e)) * g[t, slot].unsqueeze(1))
    return y


def _exact_rows(x, codes, scale, zero):
    """Group by group: scale * (the codes' product - zero point * the sum of x)."""
    y = torch.zeros((x.shape[0], codes.shape[0]), dtype=torch.float64, device=x.device)
    half = codes.shape[1] // scale.shape[1]
    for j in range(scale.shape[1]):
        c = codes[:, j * half:(j + 1) * half]
        xj = x[:, 2 * j * half:2 * (j + 1) * half]
        z = 8.0 if zero is None else zero[:, j].double()
        dot = torch.zeros_like(y)
        for o in range(8):
            byte = 2 * (o % 2) + o // 4
            nibble = c[:, byte::4] // 16 if o % 4 >= 2 else c[:, byte::4] % 16
            dot += xj[:, o::8] @ nibble.double().t()
        y += scale[:, j].double() * (dot - xj.sum(dim=1, keepdim=True) * z)
    return y


def _exact_route(s):
    l = s["l"].double().cpu().numpy()
    m, e = l.shape
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    dead = np.isneginf(l)
    if s["score"] == "sigmoid":
        score = np.where(dead, 0.0, 1.0 / (1.0 + np.exp(-np.where(dead, 0.0, l))))
    else:
        top = np.where(dead.all(1), 0.0, l.max(1))[:, None]
        score = np.exp(l - top)
        score /= np.maximum(score.sum(1), 1.0)[:, None]
    key = l if s["b"] is None and (s["groups"] == 1 or s["best"] == 1) else score + (0.0 if s["b"] is None else s["b"].double().cpu().numpy())
    key = np.where(dead | np.isnan(key), -np.inf, key)
    if s["groups"] > 1:
        size = e // s["groups"]
        total = np.full((m, s["groups"]), -np.inf)
        for j in range(s["groups"]):
            best = -np.sort(-key[:, j * size:(j + 1) * size], axis=1)[:, :s["best"]]
            total[:, j] = np.where(np.isneginf(best[:, 0]), -np.inf, np.where(np.isneginf(best), 0.0, best).sum(1))
        rank = np.argsort(-total, axis=1, kind="stable")[:, :s["keep"]]
        kept = np.zeros(total.shape, bool)
        np.put_along_axis(kept, rank, True, axis=1)
        key = np.where(np.repeat(kept, size, axis=1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :s["topk"]]
    chosen = ~np.isneginf(np.take_along_axis(key, ids, 1))
    g = np.where(chosen, np.take_along_axis(score, ids, 1), 0.0)
    if s["renorm"]:
        g = g / np.maximum(g.sum(1, keepdims=True), np.finfo(np.float64).tiny)
    return np.where(chosen, ids, -1).astype(np.int32), g * s["scale"]

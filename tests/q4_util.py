"""Inputs of the 4-bit layers' GPU tests, and the comparison with the oracle."""
from __future__ import annotations

import numpy as np

from gpu_util import say, to_dev
from oracle import q4_oracle as Q
from ternary_weight_only_tern_amd import lib as L


def weights(rng, lead, n, k, group, zero, zmax=16):
    q = rng.integers(0, 16, (*lead, n, k), dtype=np.uint8)
    s = rng.uniform(0.002, 0.02, (*lead, n, k // group)).astype(np.float16)
    z = rng.integers(0, zmax, (*lead, n, k // group), dtype=np.uint8) if zero else None
    return q, s, z


def activations(rng, m, k):
    x = rng.standard_normal((m, k))
    x[:, rng.random(k) < 0.02] *= 20
    return x.astype(np.float16)


def half(a):
    import torch
    return to_dev(np.ascontiguousarray(a).view(np.uint16)).view(torch.float16)


def upload(w) -> L.Q4Matrix:
    q, s, z = w
    return L.Q4Matrix(to_dev(Q.pack(q)), half(s), None if z is None else to_dev(z))


def kind_of(out):
    return L.TERN_F32 if out == "f32" else L.TERN_F16


def check(got, y, err, out, what):
    g = got.double().cpu().numpy()
    tol = err + Q.half_step(np.abs(y) + err, out)
    bad = ~(np.abs(g - y) <= tol)
    if bad.any():
        at = [tuple(int(v) for v in i) for i in np.argwhere(bad)[:4]]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, e.g. " +
                             ", ".join(f"{i}: {g[i]} against {y[i]} +- {tol[i]}" for i in at))
    say(what, "worst share of the tolerance", float((np.abs(g - y) / tol).max()) if g.size else 0.0)


def replay_checks(call, change, outputs):
    """Captures call(stream) and replays it, each time on changed inputs, with
    eager calls and synchronisations between; every replay equals the eager
    call bitwise."""
    import torch
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call(stream.cuda_stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call(stream.cuda_stream)
    torch.cuda.synchronize()
    for rep in range(3):
        change(rep)
        call(None)
        torch.cuda.synchronize()
        want = [t.clone() for t in outputs]
        for t in outputs:
            t.fill_(-7)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(outputs, want):
            assert torch.equal(t, w), f"replay {rep} differs from the eager call"

"""tern_q4_experts on the GPU with outputs so wide that the tokens are taken in
several rounds of bounded workspace."""
import numpy as np
import pytest

from gpu_util import say
from oracle import q4_oracle as Q
from q4_util import check, upload, weights
from ternary_weight_only_tern_amd import lib as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [2, 300])
def test_rounds_of_bounded_bytes(count):
    """3000 tokens of two slots of 60001 columns need 1.4 GiB of partials: the
    rows of a call on parts of them, and the oracle's."""
    import torch
    say("rounds", count)
    rng = np.random.default_rng(count)
    m, topk, width = 3000, 2, 60001
    up, down = weights(rng, (count,), 64, 32, 32, False), weights(rng, (count,), width, 32, 32, False)
    u, d = upload(up), upload(down)
    need = L.load().tern_q4_experts_workspace_bytes(u._at, d._at, m, topk)
    assert need < m * topk * width * 4 * 0.8
    x = torch.from_numpy(rng.standard_normal((m, 32)).astype(np.float16)).cuda()
    ids = torch.from_numpy(rng.integers(-1, count, (m, topk)).astype(np.int32)).cuda()
    g = torch.from_numpy(rng.random((m, topk)).astype(np.float32)).cuda()
    got = L.tern_q4_experts(u, d, x, ids, g)
    for a in range(0, m, 600):  # K is one step on every route: the sums' order does not depend on the tiles
        part = slice(a, a + 600)
        assert torch.equal(got[part], L.tern_q4_experts(u, d, x[part], ids[part], g[part]))
    cols = np.r_[0:5, width // 2, width - 5:width]
    few = tuple(None if w is None else w[:, cols] for w in down)
    edge = ((1 << 30) // (topk * (4 * width + 4 * 32)))  # the first round's tokens
    for a in (0, edge - 4, m - 8):
        part = slice(a, a + 8)
        y, err = Q.experts(up, few, 32, x[part].cpu().numpy(), ids[part].cpu().numpy(), g[part].cpu().numpy())
        check(got[part][:, cols], y, err, "f16", f"tokens from {a}")

"""block_attention at scores and values near the ends of what the types hold."""

import numpy as np
import pytest
import torch

import lossless_draft_verification_speculative_b200 as dv
from cache_helpers import DEV, DT, HALF_STEP, Paged
from oracle import cache_ref as ref

pytestmark = pytest.mark.gpu


def _attend(c, q, n, scale, dtype):
    """out and lse of packed queries, and the oracle's, sequence by sequence."""
    starts = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=DEV)
    lse = torch.full(q.shape[:-1], 77.0, device=DEV)
    out = dv.block_attention(q.to(DEV), **c.device(), q_start=starts, scale=scale, lse=lse)
    torch.cuda.synchronize()
    want = [ref.attend(q[sum(n[:b]):sum(n[:b + 1])].double().numpy(), *c.rows(b), n[b], scale)
            for b in range(len(n))]
    cat = {f: np.concatenate([getattr(r, f) for r in want]) for f in ("out", "lse", "wabs")}
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), cat


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,L,D", [([5], [1000], 16), ([300, 3], [700, 2000], 64),
                                   ([2], [40000], 128)])
@pytest.mark.parametrize("top", [1e3, 1e6, 1e7, 1e8, 5e8, 4e9, 1e20])
def test_scores_of_any_size(dtype, n, L, D, top):
    """Scores of a few levels, the highest among them `top` (the odd heads: the lowest -top): in
    float32 the levels are exact and far apart, so a row is the mean of the values of its highest
    level, whatever their size, and across moves of the maximum and joined pieces. Tolerance:
    half a step of the result; equal weights are off by equal factors, which cancel up to the
    float32 sums (n 2^-24) and a weight's half step."""
    c = Paged(L, 1, D, 16, dtype, seed=50)
    g = torch.Generator().manual_seed(51)
    for b, length in enumerate(L):  # the levels rise as the positions do
        t = torch.arange(length)
        level = (torch.randint(0, 4, (length,), generator=g) * 4 * t // (3 * length)).clamp(max=3)
        page = c.table[b, t // 16].long()
        c.k[page, t % 16] = 0.0
        c.k[page, t % 16, 0, 0] = (2.0 + 0.5 * level).to(DT[dtype])
    q = torch.zeros(sum(n), 2, D, dtype=DT[dtype])
    q[:, 0, 0], q[:, 1, 0] = 64.0, -64.0
    scale = float(np.float32(top / (64.0 * 3.5)))
    o, z, want = _attend(c, q, n, scale, dtype)
    u = HALF_STEP[dtype]
    bound = u * np.abs(want["out"]) + (u + max(L) * 2.0 ** -24) * want["wabs"]
    assert (np.abs(o - want["out"]) <= 1.01 * bound).all()
    # lse: log2(e) scale, its product with the score, the sum with log2 l, log 2 and its product
    # round five times, by half of 2^-23 each of a value of this size
    assert (np.abs(z - want["lse"]) <= 6 * 2.0 ** -24 * np.abs(want["lse"])
            + 2.0 ** -20 + max(L) * 2.0 ** -24).all()

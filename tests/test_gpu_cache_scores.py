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


@pytest.mark.parametrize("B,L", [(600, 300), (1, 128 * 600)])
def test_f16_values_next_to_the_end_stay_finite(B, L):
    """Values of 65504 everywhere: a weight just above a place's middle is rounded up by 2^-11, and
    with it the mean, which f16 would make infinite from 65520 on. In every fourth tile, and in
    the second after it, one key stands out, the latter by 7 binary orders and a little (below the
    8 that move the kept maximum); whole items and joined ones."""
    D = 16
    c = Paged([L], 1, D, 128, "f16", seed=52)
    c.v[c.v == c.v] = 65504.0
    c.k[c.k == c.k] = 0.0
    t = torch.arange(L)
    page = c.table[0, t // 128].long()
    c.k[page, t % 128, 0, 0] = -8.0
    one, two = (t % 512 == 5), (t % 512 == 2 * 128 + 9)
    c.k[page[one], t[one] % 128, 0, 0] = 0.0
    c.k[page[two], t[two] % 128, 0, 0] = 1.0
    d = c.device()
    d.update(page_table=d["page_table"].repeat(B, 1),
             kv_len=torch.full((B,), L, dtype=torch.int32, device=DEV))
    q = torch.zeros(B, 1, 2, D, dtype=torch.float16, device=DEV)
    q[..., 0] = 1.0
    # 2^f for f between 0 and 2^-9 covers both sides of the middle between 1 and the next f16 value
    for f in np.arange(0.0, 2.0 ** -9, 2.0 ** -14):
        out = dv.block_attention(q, **d, scale=float((7 + f) * np.log(2.0)))
        assert torch.isfinite(out).all(), f
        # a weight's half step, and the result's
        assert ((out.double() - 65504.0).abs() <= 65504.0 * 2.02 * 2.0 ** -11).all(), f
    # an infinite value that a row sees still shows
    c.v[page[5], 5, 0, 3] = float("inf")
    d["v_pages"] = c.device()["v_pages"]
    out = dv.block_attention(q, **d, scale=float(7 * np.log(2.0)))
    torch.cuda.synchronize()
    assert not torch.isfinite(out[..., 3]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("orders", [12.3, 20.7, 27.6, 29.4, 33.1])
@pytest.mark.parametrize("first", [True, False])
def test_small_weights_count(dtype, orders, first):
    """One key stands out by many binary orders over 65535 equal ones, with values that make the
    result consist of these alone. Each is off by half a step of its type, relative, and in f16 by
    2^-37 of the largest weight; the sum of float32 products and the result's rounding come on top
    (an f16 result may be subnormal: half of 2^-24)."""
    L, D = 65536, 16
    c = Paged([L], 1, D, 256, dtype, seed=43)
    at = 5 if first else L - 40
    page, slot = c.table[0, at // 256].item(), at % 256
    c.k.zero_()
    c.v.fill_(16384.0)
    c.k[page, slot, 0, 0], c.v[page, slot] = 1.0, 0.0
    q = torch.zeros(1, 2, D, dtype=DT[dtype])
    q[:, :, 0] = 8.0
    o, _, want = _attend(c, q, [1], float(np.float32(orders * np.log(2.0) / 8.0)), dtype)
    u = HALF_STEP[dtype]
    weight = u + (2.0 ** (orders - 37) if dtype == "f16" else 0.0) + L * 2.0 ** -24
    assert (np.abs(o - want["out"]) <= (u + weight) * want["out"] * 1.01 + 2.0 ** -25).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("orders", [12.3, 20.7, 27.6, 29.4, 33.1])
@pytest.mark.parametrize("at", [5, 40000])
def test_small_weights_count_in_one_item(dtype, orders, at):
    """The same where one group of warps meets all 65536 keys: 256 query heads of each of 148
    sequences, one item per CTA, whose pieces have no maxima of their own."""
    B, G, L, D = 148, 256, 65536, 16
    c = Paged([L], 1, D, 256, dtype, seed=43)
    page, slot = c.table[0, at // 256].item(), at % 256
    c.k.zero_()
    c.v.fill_(16384.0)
    c.k[page, slot, 0, 0], c.v[page, slot] = 1.0, 0.0
    d = c.device()
    d.update(page_table=d["page_table"].repeat(B, 1),
             kv_len=torch.full((B,), L, dtype=torch.int32, device=DEV))
    q = torch.zeros(B, 1, G, D, dtype=DT[dtype], device=DEV)
    q[..., 0] = 8.0
    lse = torch.zeros(B, 1, G, device=DEV)
    out = dv.block_attention(q, **d, lse=lse, scale=float(np.float32(orders * np.log(2.0) / 8.0)))
    w = (L - 1) * 2.0 ** -orders
    want = 16384.0 * w / (1 + w)
    u = HALF_STEP[dtype]
    weight = u + (2.0 ** (orders - 37) if dtype == "f16" else 0.0) + L * 2.0 ** -24
    err = (out.double() - want).abs().max().item()
    assert err <= (u + weight) * want * 1.01 + 2.0 ** -25
    z = orders * np.log(2.0) + np.log1p(w)
    assert (lse.double() - z).abs().max() <= 2.0 ** -20 * z + L * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_of_minus_infinity(dtype):
    """A seen score of -inf has a weight of 0; a row that has no other gives zeros and lse -inf."""
    D, L, n = 64, 300, 3
    c = Paged([L, L], 1, D, 16, dtype, seed=44)
    g = torch.Generator().manual_seed(45)
    q = torch.randn(2 * n, 2, D, generator=g).to(DT[dtype])
    q[:, :, 0] = -1.0
    q[:n, 1, 0] = 0.5
    d = c.device()
    k = d["k_pages"]
    for b, which in ((0, range(0, L)), (1, range(0, L, 3))):
        for t in which:
            k[c.table[b, t // 16].item(), t % 16, 0, 0] = float("inf")
    starts = torch.tensor([0, n, 2 * n], dtype=torch.int32, device=DEV)
    lse = torch.zeros(2 * n, 2, device=DEV)
    out = dv.block_attention(q.to(DEV), **d, q_start=starts, lse=lse)
    torch.cuda.synchronize()
    # sequence 0: every score -inf (head 0) or +inf (head 1)
    assert (out[:n, 0] == 0).all() and torch.isneginf(lse[:n, 0]).all()
    assert not torch.isfinite(out[:n, 1]).any()
    # sequence 1: as if the keys with infinities were not there
    keep = torch.tensor([t for t in range(L) if t % 3])
    K, V = (torch.tensor(x)[:, 0] for x in c.rows(1))
    u = HALF_STEP[dtype]
    for i in range(n):
        mine = keep[keep <= L - n + i]
        w = torch.softmax(q[n + i].double() @ K[mine].T * D ** -0.5, -1)
        err = (out[n + i].double().cpu() - w @ V[mine]).abs()
        assert (err <= 1.02 * u * (w @ V[mine].abs() + (w @ V[mine]).abs()) + 2.0 ** -16).all(), i

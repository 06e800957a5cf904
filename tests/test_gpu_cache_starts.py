"""Packed rows whose starts are out of range or decrease: a sequence with well-formed bounds is
rotated, appended and attended as it is without the others, and what is not is reported."""

import numpy as np
import pytest
import torch

import lossless_draft_verification_speculative_b200 as dv
from cache_helpers import DEV, Paged

pytestmark = pytest.mark.gpu

BAD = dv.SEQ_BAD_PARAM


def _call(starts, N, seed=0, Hq=2, Hk=1, D=16, ps=8):
    """rotary_append on packed rows with these starts; per sequence the rows of its bounds (None:
    bounds out of order or range) and what a block call of the well-formed sequences gives."""
    B = len(starts) - 1
    mine = [range(a, z) if 0 <= a <= z <= N else None for a, z in zip(starts, starts[1:])]
    n = [len(r) if r is not None else 0 for r in mine]
    kv_len = [x + 3 + b % 5 for b, x in enumerate(n)]
    g = torch.Generator().manual_seed(seed)
    x = {h: torch.randn(N, heads, D, generator=g).to(torch.bfloat16).to(DEV)
         for h, heads in (("q", Hq), ("k", Hk), ("v", Hk))}
    f = dv.rotary_frequencies(D)[0].to(DEV)
    c = Paged(kv_len, Hk, D, ps, "bf16", seed=seed)
    got, want = c.device(), c.device()
    out = torch.full_like(x["q"], 77.0)
    status = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    dv.rotary_append(x["q"], x["k"], x["v"], **got, inv_freq=f, out=out, status=status,
                     q_start=torch.tensor(starts, dtype=torch.int32, device=DEV))
    block = {h: torch.zeros(B, max(n + [1]), *t.shape[1:], dtype=t.dtype, device=DEV)
             for h, t in x.items()}
    for b, r in enumerate(mine):
        if r is not None and len(r):
            for h in x:
                block[h][b, :n[b]] = x[h][r.start:r.stop]
    qr = dv.rotary_append(block["q"], block["k"], block["v"], **want, inv_freq=f,
                          n_new=torch.tensor(n, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    return c, mine, got, want, out, qr, status.tolist(), x, n


def _pages(c, pools, b):
    """The cached keys and values of sequence b, NaN as 99."""
    ids = [int(p) for p in c.table[b] if p >= 0]
    return torch.stack([pools[k][ids] for k in ("k_pages", "v_pages")]).nan_to_num(99.0)


@pytest.mark.parametrize("starts,N", [
    ([0, 4, 8, -1, 12, 16], 16),                       # two good sequences before a bad start
    ([0, 4, 2, 30, 21, 25], 20),
    ([100, 4, 8, 9], 12),                              # the first start is too large
    ([0, 4, 8, 12, -7], 14),                           # the last one negative
    ([0, 4, 2**31 - 1, 8, 12, 12, 16], 16), ([0, 0, -2**31, 3, 3, 7], 9),
    ([0] + [3] * 20 + [1000] + list(range(3, 43)), 50),  # a search of two steps
    (list(range(0, 1500)) + [-1, 1501, 1502], 1502),     # of three
])
def test_bad_starts_leave_the_other_sequences(starts, N):
    c, mine, got, want, out, qr, status, x, n = _call(starts, N, seed=len(starts))
    covered = np.zeros(N, dtype=bool)
    for b, r in enumerate(mine):
        assert status[b] == (BAD if r is None else 0), b
        assert torch.equal(_pages(c, got, b), _pages(c, want, b)), b
        if r is not None and len(r):
            covered[r.start:r.stop] = True
            assert torch.equal(out[r.start:r.stop], qr[b, :n[b]]), b
    assert (out[torch.tensor(~covered, device=DEV)] == 77.0).all()
    # the attention of the same rows agrees about which sequences these are
    st = torch.full((len(status),), -1, dtype=torch.int32, device=DEV)
    q = torch.where((out == 77.0), torch.zeros_like(out), out)
    o = dv.block_attention(q, **got, status=st, out=torch.full_like(q, 55.0),
                           q_start=torch.tensor(starts, dtype=torch.int32, device=DEV))
    o2 = dv.block_attention(qr, **want, n_new=torch.tensor(n, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert st.tolist() == status
    vmax = max(float(x["v"].abs().max()), float(c.v.nan_to_num(0.0).abs().max()))
    for b, r in enumerate(mine):
        if r is not None and len(r):
            # (the two calls may cut and sum differently: each is off by half a step of the
            # weights, of a sum of at most the largest value, and by half a step of its result)
            a, z = o[r.start:r.stop].double(), o2[b, :n[b]].double()
            assert ((a - z).abs() <= 2.02 * 2.0 ** -8 * (vmax + z.abs())).all(), b
    assert (o[torch.tensor(~covered, device=DEV)] == 55.0).all()


@pytest.mark.parametrize("starts,N", [([0, 4, 2, 6], 8), ([0, 8, 2, 6, 8], 8),
                                      ([0, 20, 5, 9, 3, 20, 30], 30)])
def test_shared_rows_are_reported(starts, N):
    """Where starts decrease two sequences can claim one row: a sequence whose status is 0 has all
    of its rows appended, every appended slot holds its own sequence's row, and the sequence with
    the decreasing start is reported."""
    c, mine, got, want, out, qr, status, x, n = _call(starts, N)
    g0 = c.device()
    for b, r in enumerate(mine):
        assert status[b] in (0, BAD) and (r is not None or status[b] == BAD)
        have, all_, none = (_pages(c, p, b) for p in (got, want, g0))
        if status[b] == 0:
            assert torch.equal(have, all_), b
        else:
            assert ((have == all_) | (have == none)).all(), b
    for i in range(N):  # a row turned for one of its claimants, or left
        rows = [qr[b, i - r.start] for b, r in enumerate(mine) if r is not None and i in r]
        assert any(torch.equal(out[i], y) for y in rows) if rows else (out[i] == 77.0).all(), i

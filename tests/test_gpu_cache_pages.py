"""Bad page ids at every place of a tile: exactly the tokens that see the page give NaN."""

import pytest
import torch

import lossless_draft_verification_speculative_b200 as dv
from cache_helpers import DEV, Paged, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ps,L,window", [(16, 300, 40), (16, 300, None), (8, 257, 1),
                                         (64, 512, 130)])
@pytest.mark.parametrize("D,Hq", [(64, 1), (128, 4)])
def test_each_bad_page_reaches_the_tokens_that_see_it(ps, L, window, D, Hq):
    """One sequence per page, on the same pages but for that one, whose id is out of range."""
    c = Paged([L], 1, D, ps, "bf16", seed=60)
    d = c.device()
    pages = -(-L // ps)
    table = d["page_table"].repeat(pages, 1)
    for j in range(pages):
        table[j, j] = (c.n_pages, -1, 2**31 - 1, -2**31)[j % 4]
    q = queries([L], Hq, D, "bf16")[0].to(DEV)
    want = dv.block_attention(q[None], **d, window=window)[0]
    d.update(page_table=table, kv_len=torch.full((pages,), L, dtype=torch.int32, device=DEV))
    status = torch.zeros(pages, dtype=torch.int32, device=DEV)
    out = dv.block_attention(q.expand(pages, -1, -1, -1).contiguous(), **d, window=window,
                             status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [dv.SEQ_BAD_PAGE] * pages
    t = torch.arange(L, device=DEV)
    lo = torch.zeros_like(t) if window is None else (t - window + 1).clamp(min=0)
    j = torch.arange(pages, device=DEV)[:, None]
    hit = (t >= j * ps) & (lo < (j + 1) * ps)                       # [pages, L]
    assert torch.equal(out.isnan().all(-1).all(-1), hit)
    # the others: cut and summed differently, so two roundings of the weights and two of the result
    a, z = out.double(), want.double()[None]
    vmax = float(c.v.nan_to_num(0.0).abs().max())
    near = (a - z).abs() <= 2.02 * 2.0 ** -8 * (vmax + z.abs())
    assert near.all(-1).all(-1)[~hit].all()

"""A block_attention that gives up on a wait says so: every sequence's status, and NaN rather than
an earlier call's partial results where pieces are missing."""

import pytest
import torch

import lossless_draft_verification_speculative_b200 as dv
from cache_helpers import DEV, Paged, queries
from lossless_draft_verification_speculative_b200.cache import block_attention_withheld

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,L,D", [([4, 0, 2], [700, 0, 33], 128), ([200, 1], [700, 30], 64)])
def test_every_sequence_reports_it(n, L, D):
    c = Paged(L, 1, D, 16, "bf16", seed=31)
    q = torch.cat(queries(n, 4, D, "bf16")).to(DEV)
    starts = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32, device=DEV)
    d = c.device()
    ws = torch.empty(dv.block_attention_workspace_bytes(sum(n), 4, 1, D), dtype=torch.uint8,
                     device=DEV)
    status = torch.zeros(len(n), dtype=torch.int32, device=DEV)
    kw = dict(q_start=starts, workspace=ws, status=status)
    want = dv.block_attention(q, **d, **kw)     # leaves whole partial results in the workspace
    torch.cuda.synchronize()
    assert status.tolist() == [0] * len(n)
    out = torch.full_like(q, 77.0)
    block_attention_withheld(q, **d, **kw, out=out)
    torch.cuda.synchronize()
    assert status.tolist() == [dv.SEQ_TIMEOUT] * len(n)
    # every CTA's first copy was withheld, so no row is complete: unwritten, or NaN
    assert ((out == 77.0) | out.isnan()).all()
    got = dv.block_attention(q, **d, **kw)      # the same workspace, nothing withheld
    torch.cuda.synchronize()
    assert status.tolist() == [0] * len(n) and torch.equal(got, want)


def test_a_long_item_is_no_timeout():
    """One item per CTA that runs for more than a wait's limit of a second: 201326592 positions
    (every page the same), 256 rows of each of 148 heads. The keys are zeros, so every seen position
    has a score of 0 and lse is the logarithm of their number."""
    L, ps, Hk, n, D = 3 << 26, 1024, 148, 256, 16
    pages = torch.zeros(2, 1, ps, Hk, D, dtype=torch.bfloat16, device=DEV)
    pages[1, ..., :8], pages[1, ..., 8:] = 1.0, 2.0
    table = torch.zeros(1, L // ps, dtype=torch.int32, device=DEV)
    q = torch.ones(1, n, Hk, D, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lse = torch.zeros(1, n, Hk, device=DEV)
    before = dv.pipeline_timeouts()
    out = dv.block_attention(q, pages[0], pages[1], table,
                             torch.tensor([L], dtype=torch.int32, device=DEV), status=status,
                             lse=lse)
    torch.cuda.synchronize()
    assert status.tolist() == [0] and dv.pipeline_timeouts() == before
    assert torch.isfinite(out).all()
    seen = torch.arange(L - n + 1, L + 1, device=DEV).double().log()[None, :, None]
    # the sum's last additions and the logarithm: a few float32 steps of 19
    assert ((lse.double() - seen).abs() <= 2.0 ** -18).all()

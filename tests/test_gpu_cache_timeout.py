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

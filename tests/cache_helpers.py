"""Shared helpers of the cache-side GPU tests: seeded paged caches on the device, and the
derived tolerances against the float64 oracle."""

import numpy as np
import torch

import lossless_draft_verification_speculative_b200 as dv
from oracle import cache_ref as ref

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # of a rounding to the type, relative


class Paged:
    """B sequences of kv_len tokens in shuffled pages: host float64 copies of what the device
    holds. Slots behind a sequence's end, and free pages, hold NaN."""

    def __init__(self, kv_len, Hk, D, ps, dtype, seed=0, heads_first=False, extra_cols=1):
        g = torch.Generator().manual_seed(seed)
        self.kv_len, self.ps, self.dtype = list(kv_len), ps, dtype
        B = len(self.kv_len)
        need = [-(-max(0, n) // ps) for n in self.kv_len]
        self.n_pages = sum(need) + 2
        order = torch.randperm(self.n_pages, generator=g).tolist()
        cols = max(need + [1]) + extra_cols
        self.table = torch.full((B, cols), -7, dtype=torch.int32)  # unused entries are not ids
        self.k = torch.full((self.n_pages, ps, Hk, D), float("nan"), dtype=DT[dtype])
        self.v = self.k.clone()
        at = 0
        for b in range(B):
            for j in range(need[b]):
                page = order[at]
                at += 1
                self.table[b, j] = page
                m = min(ps, self.kv_len[b] - j * ps)
                self.k[page, :m] = torch.randn(m, Hk, D, generator=g).to(DT[dtype])
                self.v[page, :m] = torch.randn(m, Hk, D, generator=g).to(DT[dtype])
        self.heads_first = heads_first

    def device(self, dev=DEV):
        def put(x):
            if self.heads_first:  # [pages, heads, slots, head_dim] storage
                return x.transpose(1, 2).contiguous().to(dev).transpose(1, 2)
            return x.to(dev)
        return dict(k_pages=put(self.k), v_pages=put(self.v), page_table=self.table.to(dev),
                    kv_len=torch.tensor(self.kv_len, dtype=torch.int32, device=dev))

    def rows(self, b):
        L = self.kv_len[b]
        return (ref.gather(self.k.double().numpy(), self.table[b].numpy(), L),
                ref.gather(self.v.double().numpy(), self.table[b].numpy(), L))


def attention_bounds(r, dtype):
    """(bound of out, bound of lse) for an oracle result.

    A weight is e^z / sum: its relative error is at most twice that of e^z (numerator and sum).
    z: D products summed in float32 (D 2^-24 sum |q k|, at most 128 2^-24 qk) and the product
    with scale log2(e) (|z| 2^-23, |z| <= qk); 2^x on the SFU 2^-22 (its documented maximum) with
    the argument's own rounding, |x| 2^-24 ln 2 <= qk 2^-23; the sums and the rescalings of up to
    seen terms, (seen + 64) 2^-24. The rounded weight adds half a step of its type, and out's
    own rounding half a step of the result (subnormal f16 results: half of 2^-24)."""
    u = HALF_STEP[dtype]
    e = 2 * (r.qk * (128 + 4) * 2.0 ** -24 + 2.0 ** -21) + \
        (r.seen[:, None] + 64) * 2.0 ** -24
    e = e[..., None]
    out = (u + e) * r.wabs * (1 + u) + u * np.abs(r.out) + 2.0 ** -25
    with np.errstate(invalid="ignore"):
        lse = e[..., 0] + 2.0 ** -22 * np.where(np.isfinite(r.lse), np.abs(r.lse), 0.0) + 2.0 ** -22
    return out, lse


def check_attention(cache, q, n_new, dtype, *, packed=False, scale=None, causal=True, window=None,
                    N=None, out=None, **kw):
    """Run block_attention on cache (Paged) with q, a list of [n, Hq, D] per sequence, and compare
    every row with the oracle; rows of no sequence must keep what they held. Returns out, lse."""
    B, (_, Hq, D) = len(n_new), q[0].shape
    N = max(n_new + [1]) if N is None else N
    d = cache.device()
    if packed:
        qs = torch.cat(q + [torch.full((3, Hq, D), 5.0, dtype=DT[dtype])])
        starts = torch.tensor(np.concatenate([[0], np.cumsum(n_new)]), dtype=torch.int32)
        form = dict(q_start=starts.to(DEV))
        where = [(slice(int(starts[b]), int(starts[b + 1])),) for b in range(B)]
    else:
        qs = torch.full((B, N, Hq, D), float("nan"), dtype=DT[dtype])
        for b in range(B):
            qs[b, :n_new[b]] = q[b]
        form = dict(n_new=torch.tensor(n_new, dtype=torch.int32, device=DEV))
        where = [(b, slice(0, n_new[b])) for b in range(B)]
    if out is None:
        out = torch.empty(qs.shape, dtype=DT[dtype], device=DEV)
    out.fill_(77.0)
    lse = torch.full(qs.shape[:-1], 77.0, device=DEV)
    status = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    before = dv.pipeline_timeouts()
    got = dv.block_attention(qs.to(DEV), **d, **form, scale=scale, causal=causal, window=window,
                             out=out, lse=lse, status=status, **kw)
    torch.cuda.synchronize()
    assert got is out and dv.pipeline_timeouts() == before
    assert status.tolist() == [0] * B
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    mine = np.zeros(o.shape[:-2], dtype=bool)
    for b in range(B):
        mine[where[b]] = True
        K, V = cache.rows(b)
        r = ref.attend(q[b].double().numpy(), K, V, n_new[b],
                       D ** -0.5 if scale is None else scale, causal, window)
        bo, bz = attention_bounds(r, dtype)
        eo = np.abs(o[where[b]] - r.out)
        assert (eo <= bo).all(), (b, float((eo / bo).max()))
        seen = np.isfinite(r.lse)
        assert np.array_equal(np.isneginf(z[where[b]]), ~seen), b
        assert (np.abs(z[where[b]] - r.lse)[seen] <= bz[seen]).all(), b
        assert (o[where[b]][~seen] == 0).all()
    assert (o[~mine] == 77.0).all() and (z[~mine] == 77.0).all()
    return out, lse


def queries(n_new, Hq, D, dtype, seed=0, size=2.0):
    g = torch.Generator().manual_seed(1000 + seed)
    return [(size * torch.randn(n, Hq, D, generator=g)).to(DT[dtype]) for n in n_new]

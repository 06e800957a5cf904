"""The cache-side operators on the GPU against the float64 oracle (tolerances derived in
``cache_helpers.py`` and below, before their first run)."""

import numpy as np
import pytest
import torch

import lossless_draft_verification_speculative_b200 as dv
from cache_helpers import (DEV, DT, HALF_STEP, Paged, attention_bounds, check_attention, queries)
from oracle import cache_ref as ref

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------- block attention

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hk,D,ps", [(8, 2, 128, 16), (4, 4, 64, 32), (7, 1, 128, 64),
                                        (10, 2, 64, 8), (6, 2, 80, 16), (2, 1, 16, 16),
                                        (4, 2, 96, 128), (5, 5, 72, 256), (33, 1, 120, 1024)])
def test_head_layouts(dtype, Hq, Hk, D, ps):
    """Verify blocks of 1 to 9 tokens over caches that end inside pages and tiles."""
    n = [1, 9, 4, 3]
    c = Paged([1, 200, 128, 387], Hk, D, ps, dtype, seed=D + ps)
    check_attention(c, queries(n, Hq, D, dtype), n, dtype)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("causal,window", [(True, None), (False, None), (True, 1), (True, 100),
                                           (False, 7), (False, 300)])
def test_masks(packed, causal, window):
    n = [5, 0, 8, 1, 7]
    c = Paged([5, 0, 300, 129, 640], 2, 64, 16, "bf16", seed=3)
    check_attention(c, queries(n, 8, 64, "bf16"), n, "bf16", packed=packed, causal=causal,
                    window=window)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 383, 385, 1000])
def test_lengths_around_pages_and_tiles(L):
    n = [1, min(L, 3)]
    c = Paged([L, L], 1, 128, 16, "f16", seed=L)
    check_attention(c, queries(n, 4, 128, "f16"), n, "f16")


@pytest.mark.parametrize("n,Hq,Hk,L", [(15, 8, 1, 500), (16, 8, 1, 500), (17, 8, 1, 500),
                                       (33, 8, 1, 700), (128, 2, 1, 128), (129, 2, 2, 400),
                                       (257, 3, 1, 300), (300, 2, 1, 900), (40, 12, 2, 129)])
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(n, Hq, Hk, L, causal):
    """Chunks of prompts: rows that fill one or two query tiles, and more, exactly or not."""
    c = Paged([L, n], Hk, 64, 64, "bf16", seed=n)
    check_attention(c, queries([n, n], Hq, 64, "bf16"), [n, n], "bf16", packed=True, causal=causal)


def test_chunk_of_wide_heads():
    n = [300, 1, 70]
    c = Paged([1111, 400, 70], 2, 128, 32, "f16", seed=9)
    check_attention(c, queries(n, 8, 128, "f16"), n, "f16", packed=True)
    check_attention(c, queries(n, 8, 128, "f16"), n, "f16", packed=True, window=200)


def test_rows_that_see_nothing():
    """A cache shorter than the block (its first tokens lie before position 0), and empty ones."""
    n = [4, 3, 2]
    c = Paged([2, 0, 0], 1, 64, 16, "bf16", seed=4)
    check_attention(c, queries(n, 2, 64, "bf16"), n, "bf16")
    check_attention(c, queries(n, 2, 64, "bf16"), n, "bf16", causal=False)
    n = [200]
    c = Paged([30], 1, 64, 16, "bf16", seed=4)  # a whole query tile before position 0
    check_attention(c, queries(n, 2, 64, "bf16"), n, "bf16")


def test_many_sequences_of_one_token():
    rng = np.random.default_rng(5)
    L = rng.integers(0, 90, 700).tolist()
    n = [min(1, x) for x in L]
    c = Paged(L, 1, 16, 8, "bf16", seed=5)
    check_attention(c, queries(n, 1, 16, "bf16"), n, "bf16")


def test_long_context_is_split_and_joined():
    n = [3, 1]
    c = Paged([30011, 9], 1, 64, 64, "bf16", seed=6)
    check_attention(c, queries(n, 4, 64, "bf16"), n, "bf16")


def test_heads_first_storage_and_strided_rows():
    """[pages, heads, slots, head_dim] storage; q a slice of fused projections; a strided out."""
    n = [2, 6]
    c = Paged([100, 333], 2, 64, 16, "bf16", seed=7, heads_first=True)
    q = queries(n, 4, 64, "bf16")
    check_attention(c, q, n, "bf16")
    wide = torch.empty(2, 6, 8, 64, dtype=torch.bfloat16, device=DEV)
    check_attention(c, q, n, "bf16", out=wide[:, :, 2:6])
    fused = torch.full((2, 6, 8, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    for b in range(2):
        fused[b, :n[b], 3:7] = q[b].to(DEV)
    kw = dict(n_new=torch.tensor(n, dtype=torch.int32, device=DEV))
    a = dv.block_attention(fused[:, :, 3:7], **c.device(), **kw)
    b = dv.block_attention(fused[:, :, 3:7].contiguous(), **c.device(), **kw)
    for i in range(2):
        assert torch.equal(a[i, :n[i]], b[i, :n[i]])


def test_layouts_of_keys_beside_values():
    """Values before keys in memory, both in one tensor, and keys and values of different
    strides give what two plain tensors give."""
    n = [3, 5]
    c = Paged([70, 200], 2, 64, 16, "bf16", seed=40)
    q = torch.full((2, 5, 4, 64), 1.0, dtype=torch.bfloat16, device=DEV)
    for b, x in enumerate(queries(n, 4, 64, "bf16")):
        q[b, :n[b]] = x.to(DEV)
    kw = dict(n_new=torch.tensor(n, dtype=torch.int32, device=DEV))
    d = c.device()
    want = dv.block_attention(q, **d, **kw, out=torch.zeros_like(q))
    pair = torch.stack([d["v_pages"], d["k_pages"]])                     # values first
    inner = torch.stack([d["k_pages"], d["v_pages"]], dim=1)             # page by page
    mixed = d["v_pages"].transpose(1, 2).contiguous().transpose(1, 2)    # other strides
    for k, v in ((pair[1], pair[0]), (inner[:, 0], inner[:, 1]), (d["k_pages"], mixed),
                 (mixed, mixed)):
        got = dv.block_attention(q, **{**d, "k_pages": k, "v_pages": v}, **kw,
                                 out=torch.zeros_like(q))
        if k is v:  # keys that are the values: another result, but a defined one
            want = dv.block_attention(q, **{**d, "k_pages": d["v_pages"]}, **kw,
                                      out=torch.zeros_like(q))
        assert torch.equal(got, want)


def test_scale_and_large_scores():
    """Peaked rows (scores of hundreds): the running maximum moves, nothing overflows."""
    n = [4]
    c = Paged([600], 1, 64, 16, "bf16", seed=8)
    check_attention(c, queries(n, 2, 64, "bf16", size=20.0), n, "bf16", scale=1.0)
    c.k[c.table[0, 37].item(), :8] *= 8  # the largest scores come last
    check_attention(c, queries(n, 2, 64, "bf16", size=8.0), n, "bf16", scale=0.5)
    check_attention(c, queries(n, 2, 64, "bf16"), n, "bf16", scale=1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("orders", [17.5, 25.5, 28.0])
def test_many_small_weights(dtype, orders):
    """One key stands out by many binary orders over 65535 equal ones, whose sum still counts."""
    L, D = 65536, 16
    c = Paged([L], 1, D, 256, dtype, seed=42)
    c.k.zero_()
    c.v.fill_(1.0)
    c.k[c.table[0, 0].item(), 5, 0, 0] = 1.0
    q = torch.zeros(1, 2, D, dtype=DT[dtype])
    q[:, :, 0] = 8.0
    check_attention(c, [q], [1], dtype, scale=orders * np.log(2.0) / 8.0)


@pytest.mark.parametrize("n,Hq", [([8], 4), ([100, 8], 4)])
def test_unseen_places_hold_anything(n, Hq):
    """Infinities and NaN in the cache where a token does not look (later tokens of its own
    block, before its window) leave its result as it was; where it looks, the element is not
    finite."""
    D, L = 64, [300, 290][:len(n)]
    c = Paged(L, 1, D, 16, "bf16", seed=10)
    q = queries(n, Hq, D, "bf16")
    out0, lse0 = check_attention(c, q, n, "bf16", packed=True, window=120)
    bad = L[0] - 3          # one of the block's own tokens
    page, slot = c.table[0, bad // 16].item(), bad % 16
    early = 20              # before every token's window
    pe, se = c.table[0, early // 16].item(), early % 16
    for kval, vval in ((float("nan"), 1.0), (1.0, float("nan")), (0.5, float("inf"))):
        c2 = Paged(L, 1, D, 16, "bf16", seed=10)
        c2.k[page, slot, 0, 3], c2.v[page, slot, 0, 5] = kval, vval
        c2.k[pe, se], c2.v[pe, se] = float("inf"), float("nan")
        d = c2.device()
        starts = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=DEV)
        out = dv.block_attention(torch.cat(q).to(DEV), **d, q_start=starts, window=120)
        torch.cuda.synchronize()
        keep = n[0] - 3     # tokens before the bad position
        assert torch.equal(out[:keep], out0[:keep])
        assert torch.equal(out[n[0]:sum(n)], out0[n[0]:sum(n)])
        hit = out[keep:n[0]]
        assert not torch.isfinite(hit[..., 5]).any()


def test_bad_parameters_and_pages():
    """Counts, starts, lengths and page ids out of range: nothing out of range is touched, the
    sequence is reported, the others are right."""
    Hq, D = 4, 64
    c = Paged([100, 60, 300, 40, 20], 2, D, 16, "bf16", seed=11)
    q = torch.cat([x[None] for x in queries([4] * 5, Hq, D, "bf16")]).to(DEV)
    d = c.device()
    good = dv.block_attention(q, **d)
    d["kv_len"] = torch.tensor([100, -1, 300, 16 * c.table.shape[1] + 1, 20], dtype=torch.int32,
                               device=DEV)
    n = torch.tensor([4, 4, 5, 4, -2], dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 55.0)
    status = torch.zeros(5, dtype=torch.int32, device=DEV)
    dv.block_attention(q, **d, n_new=n, out=out, status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 16, 16, 16, 16]
    assert torch.equal(out[0], good[0]) and (out[1:] == 55.0).all()
    # bad pages: a token that sees one gives NaN, a token that does not is right
    d = c.device()
    d["page_table"][0, 1] = c.n_pages         # positions 16..31 of sequence 0
    d["page_table"][2, 18] = -1               # positions 288..303: the last ones of sequence 2
    d["page_table"][4, 1] = 1 << 30           # positions 16..31 of sequence 4
    out = dv.block_attention(q, **d, status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [32, 0, 32, 0, 32]
    assert torch.isnan(out[0]).all() and torch.isnan(out[2]).all()
    assert torch.equal(out[1], good[1]) and torch.equal(out[3], good[3])
    assert torch.isnan(out[4]).all()          # positions 16..19 are its own tokens
    out = dv.block_attention(q, **d, status=status, window=50)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0, 32, 0, 32]  # sequence 0's window no longer reaches it
    ok = dv.block_attention(q, **c.device(), window=50)
    assert torch.equal(out[0], ok[0]) and torch.isnan(out[2]).all()
    # packed starts
    starts = torch.tensor([0, 4, 2, 30, 21, 25], dtype=torch.int32, device=DEV)
    out = torch.full((20, Hq, D), 55.0, dtype=torch.bfloat16, device=DEV)
    dv.block_attention(q.view(20, Hq, D), **c.device(), q_start=starts, out=out, status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 16, 16, 16, 16]
    assert torch.equal(out[:4], good[0]) and (out[4:] == 55.0).all()


@pytest.mark.parametrize("n,L", [([4, 2], [900, 33]), ([300], [700])])
def test_result_over_the_queries(n, L):
    """out may be q itself, for whole items and for ones that several CTAs share."""
    c = Paged(L, 2, 64, 16, "bf16", seed=41)
    q = torch.cat(queries(n, 8, 64, "bf16")).to(DEV)
    starts = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=DEV)
    want = dv.block_attention(q, **c.device(), q_start=starts)
    got = dv.block_attention(q, **c.device(), q_start=starts, out=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(got, want)


def test_empty_calls():
    c = Paged([30], 1, 64, 16, "bf16")
    d = c.device()
    q = torch.zeros(1, 0, 2, 64, dtype=torch.bfloat16, device=DEV)
    status = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    assert dv.block_attention(q, **d, status=status).shape == q.shape
    assert status.item() == 0
    d = {k: (v[:0] if k in ("page_table", "kv_len") else v) for k, v in d.items()}
    assert dv.block_attention(q[:0], **d).shape == (0, 0, 2, 64)


def test_repeats_bit_for_bit_and_on_a_side_stream():
    n = [8] * 12
    c = Paged(list(range(500, 3500, 250)), 2, 128, 64, "bf16", seed=12)
    q = torch.cat([x[None] for x in queries(n, 8, 128, "bf16")]).to(DEV)
    d = c.device()
    a = dv.block_attention(q, **d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = dv.block_attention(q, **d)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_two_calls_at_once():
    """Calls that overlap on two streams have their own workspaces."""
    cs = [Paged([5000, 4000 + 900 * i], 1, 64, 16, "bf16", seed=20 + i) for i in range(2)]
    qs = [torch.cat([x[None] for x in queries([4, 4], 4, 64, "bf16", seed=i)]).to(DEV)
          for i in range(2)]
    ds = [c.device() for c in cs]
    want = [dv.block_attention(q, **d) for q, d in zip(qs, ds)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(dv.block_attention(qs[i], **ds[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("n,D", [(4, 128), (200, 64)])
def test_timeout_path(n, D):
    """With every CTA's first copy of keys withheld the waits for it run out: the kernel gives up
    and frees what it holds, the counter grows, and the next call is right."""
    from lossless_draft_verification_speculative_b200.cache import block_attention_withheld

    c = Paged([700], 1, D, 16, "bf16", seed=30)
    q = queries([n], 4, D, "bf16")
    before = dv.pipeline_timeouts()
    block_attention_withheld(q[0][None].to(DEV), **c.device())
    torch.cuda.synchronize()
    assert dv.pipeline_timeouts() > before
    check_attention(c, q, [n], "bf16")


# --------------------------------------------------------------------------- rotary append

def check_rotary(kv_len, n_new, Hq, Hk, D, R, ps, dtype, *, interleaved=False, packed=False,
                 magnitude=1.0, theta=10000.0, in_place=False, aligned=True, seed=0, N=None):
    """Every query and every page element against the oracle: an output of the rotation is
    within half a step of its type of the float64 value, plus 2^-21 (|x1| + |x2|) for the float32
    sine, cosine (each within 2^-22: the reduced angle rounds at 2^-25 of a turn, sincospi at two
    steps) and products; copied elements are equal; other slots keep what they held."""
    B, g = len(kv_len), torch.Generator().manual_seed(seed)
    c = Paged(kv_len, Hk, D, ps, dtype, seed=seed)
    T = sum(n_new)
    x = {h: [torch.randn(n, heads, D, generator=g).to(DT[dtype]) for n in n_new]
         for h, heads in (("q", Hq), ("k", Hk), ("v", Hk))}
    f = torch.tensor(ref.frequencies(R, theta)[0], dtype=torch.float32) if R else None
    N = max(n_new + [1]) if N is None else N
    dev = {}
    for h, heads in (("q", Hq), ("k", Hk), ("v", Hk)):
        if packed:
            t = torch.cat(x[h] + [torch.full((2, heads, D), 5.0, dtype=DT[dtype])])
        else:
            t = torch.full((B, N, heads, D), 5.0, dtype=DT[dtype])
            for b in range(B):
                t[b, :n_new[b]] = x[h][b]
        if not aligned:  # rows that start on odd elements
            wide = torch.zeros(*t.shape[:-1], D + 1, dtype=DT[dtype], device=DEV)
            wide[..., 1:] = t.to(DEV)
            dev[h] = wide[..., 1:]
        else:
            dev[h] = t.to(DEV)
    starts = [sum(n_new[:b]) for b in range(B + 1)]
    form = dict(q_start=torch.tensor(starts, dtype=torch.int32, device=DEV)) if packed else \
        dict(n_new=torch.tensor(n_new, dtype=torch.int32, device=DEV))
    out = dev["q"] if in_place else torch.full(dev["q"].shape, 77.0, dtype=DT[dtype], device=DEV)
    d = c.device()
    status = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    got = dv.rotary_append(dev["q"], dev["k"], dev["v"], **d, inv_freq=None if f is None else
                           f.to(DEV), **form, interleaved=interleaved, magnitude=magnitude,
                           out=out, status=status)
    torch.cuda.synchronize()
    assert got is out and status.tolist() == [0] * B
    u = HALF_STEP[dtype]
    freq = f.double().numpy() if R else np.zeros(0)
    want_k, want_v = c.k.double().numpy(), c.v.double().numpy()
    tol_k = np.zeros_like(want_k)
    o = out.double().cpu().numpy()
    mine = np.zeros(o.shape[:-2], dtype=bool)
    for b in range(B):
        for i in range(n_new[b]):
            p = kv_len[b] - n_new[b] + i
            at = (starts[b] + i,) if packed else (b, i)
            mine[at] = True
            y, size = ref.rotate(x["q"][b][i].double().numpy(), p, freq, interleaved, magnitude)
            tol = (size > 0) * (u * np.abs(y) + 2.0 ** -21 * size + 2.0 ** -25)
            assert (np.abs(o[at] - y) <= tol).all(), (b, i)
            y, size = ref.rotate(x["k"][b][i].double().numpy(), p, freq, interleaved, magnitude)
            page, slot = int(c.table[b, p // ps]), p % ps
            want_k[page, slot] = y
            tol_k[page, slot] = (size > 0) * (u * np.abs(y) + 2.0 ** -21 * size + 2.0 ** -25)
            want_v[page, slot] = x["v"][b][i].double().numpy()
    k, v = d["k_pages"].double().cpu().numpy(), d["v_pages"].double().cpu().numpy()
    live = ~np.isnan(want_k)
    assert np.array_equal(np.isnan(k), ~live) and np.array_equal(np.isnan(v), ~live)
    assert (np.abs(k - want_k)[live] <= tol_k[live]).all()
    assert np.array_equal(v[live], want_v[live])
    assert (o[~mine] == (5.0 if in_place else 77.0)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (64, 64), (64, 16), (80, 80), (80, 32),
                                 (72, 24), (96, 0), (6, 4), (17, 10), (256, 256)])
def test_rotary_heads(dtype, interleaved, D, R):
    n = [1, 6, 0, 3]
    check_rotary([1, 50, 7, 33], n, 5, 2, D, R, 16, dtype, interleaved=interleaved, seed=D + R)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(in_place=True), dict(aligned=False),
                                dict(magnitude=1.25), dict(interleaved=True, aligned=False)])
def test_rotary_forms(packed, kw):
    check_rotary([10, 40, 3, 64], [10, 1, 3, 17], 4, 1, 64, 64, 8, "bf16", packed=packed, **kw)


def test_rotary_far_positions():
    """Positions near 2^20 with a frequency of 1: float32 angles would be off by 0.03."""
    ps = 512
    n, L = [3], [(1 << 20) - 1]
    g = torch.Generator().manual_seed(1)
    cols = (L[0] + ps - 1) // ps
    table = torch.full((1, cols), -1, dtype=torch.int32)
    table[0, -1] = 0
    q = torch.randn(1, 3, 2, 64, generator=g).to(torch.float16)
    f = torch.tensor(ref.frequencies(64, 10000.0)[0], dtype=torch.float32)
    pages = torch.zeros(1, ps, 2, 64, dtype=torch.float16, device=DEV)
    out = dv.rotary_append(q.to(DEV), q.to(DEV), q.to(DEV), pages, pages.clone(), table.to(DEV),
                           torch.tensor(L, dtype=torch.int32, device=DEV), f.to(DEV))
    torch.cuda.synchronize()
    for i in range(3):
        p = L[0] - 3 + i
        y, size = ref.rotate(q[0, i].double().numpy(), p, f.double().numpy())
        tol = 2.0 ** -11 * np.abs(y) + 2.0 ** -21 * size + 2.0 ** -25
        assert (np.abs(out[0, i].double().cpu().numpy() - y) <= tol).all()
        assert torch.equal(pages[0, p % ps], out[0, i])


def test_rotary_many_tokens_and_sequences():
    """Several tokens a CTA (a long prompt), and a search over many packed starts."""
    check_rotary([700, 6000], [600, 4600], 1, 1, 16, 16, 64, "bf16", packed=True, seed=3)
    rng = np.random.default_rng(3)
    n = rng.integers(0, 3, 1500).tolist()
    check_rotary([max(x, 1) for x in n], n, 1, 1, 16, 16, 8, "f16", packed=True, seed=4)


def test_rotary_bad_parameters_and_pages():
    Hk, D = 1, 64
    c = Paged([10, 20, 30, 40, 2], Hk, D, 16, "bf16", seed=5)
    d = c.device()
    q = torch.randn(5, 3, 2, D, device=DEV).to(torch.bfloat16)
    k = torch.randn(5, 3, Hk, D, device=DEV).to(torch.bfloat16)
    f = torch.ones(D // 2, device=DEV)
    d["kv_len"][1] = -4
    d["page_table"][2, 1] = c.n_pages         # the new tokens of sequence 2
    d["page_table"][3, 0] = -1                # not where sequence 3 appends
    n = torch.tensor([3, 3, 3, 4, 3], dtype=torch.int32, device=DEV)  # 4 > N; 3 > kv_len[4]
    status = torch.zeros(5, dtype=torch.int32, device=DEV)
    out = torch.full_like(q, 55.0)
    k0 = d["k_pages"].clone()
    dv.rotary_append(q, k, k, **d, inv_freq=f, n_new=n, out=out, status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 16, 32, 16, 16]
    assert (out[[1, 3, 4]] == 55.0).all() and not (out[[0, 2]] == 55.0).any()
    page = c.table[0, 0].item()
    d["k_pages"][page, 7:10] = k0[page, 7:10]  # only sequence 0 appended
    assert torch.equal(d["k_pages"].isnan(), k0.isnan())
    assert torch.equal(d["k_pages"].nan_to_num(), k0.nan_to_num())
    n[3] = 3
    dv.rotary_append(q, k, k, **d, inv_freq=f, n_new=n, out=out, status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 16, 32, 0, 16]


def test_rotary_empty_calls():
    c = Paged([30], 1, 64, 16, "bf16")
    q = torch.zeros(1, 0, 1, 64, dtype=torch.bfloat16, device=DEV)
    status = torch.full((1,), 9, dtype=torch.int32, device=DEV)
    assert dv.rotary_append(q, q, q, **c.device(), inv_freq=None, status=status).shape == q.shape
    assert status.item() == 0


# ------------------------------------------------------------------------------- together

def test_captured_cycle_replays_on_new_lengths():
    """rotary_append and block_attention captured into one graph: replayed after the lengths, the
    counts and the values in the same buffers have changed, it gives what eager calls give."""
    B, N, Hq, Hk, D, ps = 3, 4, 4, 2, 64, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    pool = [torch.randn(40, ps, Hk, D, generator=g, device=DEV).to(torch.bfloat16)
            for _ in range(2)]
    table = torch.arange(39, dtype=torch.int32, device=DEV).view(3, 13)
    kv_len = torch.tensor([4, 100, 60], dtype=torch.int32, device=DEV)
    n_new = torch.tensor([4, 1, 2], dtype=torch.int32, device=DEV)
    q = torch.randn(B, N, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    k = torch.randn(B, N, Hk, D, generator=g, device=DEV).to(torch.bfloat16)
    f = torch.tensor(ref.frequencies(D, 1e4)[0], dtype=torch.float32, device=DEV)
    qr, out = torch.zeros_like(q), torch.zeros_like(q)

    def cycle(pool, qr, out):
        dv.rotary_append(q, k, k, *pool, table, kv_len, f, n_new=n_new, out=qr)
        dv.block_attention(qr, *pool, table, kv_len, n_new=n_new, out=out)

    cycle([x.clone() for x in pool], qr, out)  # the first call on the device sets it up
    torch.cuda.synchronize()
    mine = [x.clone() for x in pool]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cycle(mine, qr, out)
    eager = [x.clone() for x in pool]
    for lens, counts in (([4, 100, 60], [4, 1, 2]), ([205, 9, 1], [1, 4, 0]),
                         ([130, 64, 128], [2, 3, 4])):
        kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        n_new.copy_(torch.tensor(counts, dtype=torch.int32))
        q.normal_(generator=g)
        k.normal_(generator=g)
        qr.zero_()
        out.zero_()
        graph.replay()
        a = (qr.clone(), out.clone())
        qr2, out2 = torch.zeros_like(q), torch.zeros_like(q)
        cycle(eager, qr2, out2)
        torch.cuda.synchronize()
        assert torch.equal(a[0], qr2) and torch.equal(a[1], out2)
        assert all(torch.equal(x, y) for x, y in zip(mine, eager))


def test_speculative_cycles_equal_plain_decoding():
    """Cycles of a one-layer model through rotary_append, block_attention and greedy_accept, with
    rejected drafts rolled back by kv_len, give the tokens of plain one-token decoding through
    the same two operators (whose scores are far from ties here)."""
    V, Hq, Hk, D, ps, K, B = 97, 4, 2, 64, 16, 3, 3
    g = torch.Generator(device=DEV).manual_seed(7)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV)

    emb = rnd(V, 64)
    wq, wk, wv = rnd(64, Hq * D) / 8, rnd(64, Hk * D) / 8, rnd(64, Hk * D) / 8
    wo = rnd(Hq * D, V)
    f = dv.rotary_frequencies(D, 10000.0)[0].to(DEV)
    table = torch.randperm(3 * B, generator=g, device=DEV).to(torch.int32).view(B, 3)

    def pools():
        return [torch.full((3 * B, ps, Hk, D), float("nan"), dtype=torch.bfloat16, device=DEV)
                for _ in range(2)]

    def forward(tokens, pool, kv_len, n_new=None):
        x = emb[tokens]
        n = tokens.shape[1]
        q, k, v = ((x @ w).to(torch.bfloat16).view(B, n, -1, D) for w in (wq, wk, wv))
        q = dv.rotary_append(q, k, v, *pool, table, kv_len, f, n_new=n_new)
        o = dv.block_attention(q, *pool, table, kv_len, n_new=n_new)
        return o.float().reshape(B, n, -1) @ wo

    prompt = torch.randint(0, V, (B, 5), generator=g, device=DEV)
    steps = 24

    def start():
        pool = pools()
        kv = torch.full((B,), 5, dtype=torch.int32, device=DEV)
        return pool, kv, forward(prompt, pool, kv)[:, -1].argmax(-1)

    pool, kv, tok = start()
    plain = [tok]
    for _ in range(steps):
        kv = kv + 1
        tok = forward(tok[:, None], pool, kv)[:, -1].argmax(-1)
        plain.append(tok)
    plain = torch.stack(plain, 1).tolist()

    # a drafter that is right about two times in three
    rng = np.random.default_rng(8)
    pool, kv, tok = start()
    got = [[int(t)] for t in tok]
    while min(len(x) for x in got) < steps:
        drafts = torch.tensor([[plain[b][min(len(got[b]) + i, steps)] if rng.random() < 0.67 else
                                int(rng.integers(V)) for i in range(K)] for b in range(B)],
                              dtype=torch.int32, device=DEV)
        anchor = torch.tensor([x[-1] for x in got], device=DEV)
        # the block: the anchor and its drafts; rows 0..K of the logits verify them
        kv_block = (kv + K + 1).clamp(max=3 * ps)
        logits = forward(torch.cat([anchor[:, None], drafts.long()], 1), pool, kv_block)
        r = dv.greedy_accept(logits.contiguous(), drafts)
        kv = kv + r.n_accepted + 1          # the anchor and the accepted drafts stay
        for b in range(B):
            j = int(r.n_accepted[b])
            got[b] += r.tokens[b, :j + 1].tolist()
        if int(kv.max()) + K + 1 > 3 * ps:
            break
    assert min(len(x) for x in got) >= 10
    for b in range(B):
        m = min(len(got[b]), steps)
        assert got[b][:m] == plain[b][:m]

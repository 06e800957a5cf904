"""Refusals of the cache-side calls, without a GPU: the C entry points reject bad arguments
before any CUDA call (fake device addresses, never dereferenced), and the Python wrappers reject
bad layouts before any pointer reaches the library."""

import ctypes

import pytest
import torch

import lossless_draft_verification_speculative_b200 as dv
from lossless_draft_verification_speculative_b200 import build_lib
from lossless_draft_verification_speculative_b200 import cache as ch

FAKE = 0x10000
OK, INV, UNS, WS = 0, 1, 2, 4
BF16, F32, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return ch._lib()


def _args(**kw):
    """Arguments of a valid block call: B = 4, N = 8, 8 / 2 heads of 64, pages of 16."""
    D, Hq, Hk = kw.pop("D", 64), kw.pop("Hq", 8), kw.pop("Hk", 2)
    ps = kw.pop("ps", 16)
    cache = dict(k=FAKE, v=FAKE, k_page_stride=ps * Hk * D, k_token_stride=Hk * D,
                 k_head_stride=D, v_page_stride=ps * Hk * D, v_token_stride=Hk * D,
                 v_head_stride=D, n_pages=100, page_size=ps, n_heads=Hk, head_dim=D,
                 page_table=FAKE, ld_table=10, max_pages=10, kv_len=FAKE)
    rows = dict(B=4, N=8, n_new=FAKE, q_start=None)
    q = dict(p=FAKE, seq_stride=8 * Hq * D, token_stride=Hq * D, head_stride=D)
    kv = dict(p=FAKE, seq_stride=8 * Hk * D, token_stride=Hk * D, head_stride=D)
    a = dict(q=q, out=dict(q), k=kv, v=dict(kv), cache=cache, rows=rows, Hq=Hq, dt=BF16)
    for key, val in kw.items():
        if key in a and isinstance(a[key], dict):
            a[key] = {**a[key], **val}
        else:
            a[key] = val
    return a


def _rotary(lib, **kw):
    a = dict(inv=FAKE, R=64, il=0, mag=1.0, status=None)
    a.update(_args(**kw))
    return lib.dspark_rotary_append(ch.Heads(**a["q"]), a["Hq"], ch.Heads(**a["out"]),
                                    ch.Heads(**a["k"]), ch.Heads(**a["v"]), a["dt"],
                                    ch.KvCache(**a["cache"]), ch.Rows(**a["rows"]), a["inv"],
                                    a["R"], a["il"], a["mag"], a["status"], None)


def _attend(lib, **kw):
    a = dict(scale=0.125, causal=1, window=0, lse=None, status=None, ws=FAKE, wsb=1 << 40)
    a.update(_args(**kw))
    return lib.dspark_block_attention(ch.Heads(**a["q"]), a["Hq"], ch.Heads(**a["out"]), a["dt"],
                                      ch.KvCache(**a["cache"]), ch.Rows(**a["rows"]), a["scale"],
                                      a["causal"], a["window"], a["lse"], a["status"], a["ws"],
                                      a["wsb"], None)


@pytest.mark.parametrize("call", [_rotary, _attend])
@pytest.mark.parametrize("want,kw", [
    (INV, dict(dt=F32)), (INV, dict(dt=7)),
    (INV, dict(rows=dict(B=-1))), (INV, dict(rows=dict(N=-1))),
    (INV, dict(rows=dict(q_start=FAKE))),                    # a block's counts and packed starts
    (INV, dict(Hq=0)), (INV, dict(cache=dict(n_heads=0))),
    (INV, dict(cache=dict(head_dim=0))), (INV, dict(cache=dict(page_size=0))),
    (INV, dict(cache=dict(n_pages=0))), (INV, dict(cache=dict(max_pages=-1))),
    (INV, dict(cache=dict(ld_table=9))), (INV, dict(cache=dict(page_table=None))),
    (INV, dict(cache=dict(kv_len=None))), (INV, dict(cache=dict(k=None))),
    (INV, dict(cache=dict(v=None))), (INV, dict(cache=dict(k_token_stride=63))),
    (INV, dict(cache=dict(v_head_stride=8))), (INV, dict(cache=dict(k_page_stride=-1))),
    (INV, dict(q=dict(p=None))), (INV, dict(out=dict(p=None))),
    (INV, dict(q=dict(token_stride=-8))),
    (INV, dict(out=dict(head_stride=0))), (INV, dict(out=dict(seq_stride=0))),
    (UNS, dict(D=2048)), (UNS, dict(Hq=8192, Hk=8192, ps=8)), (UNS, dict(rows=dict(B=70000))),
    (UNS, dict(rows=dict(B=60000, N=60000))),
    (UNS, dict(cache=dict(max_pages=1 << 28, ld_table=1 << 28))),
    (UNS, dict(cache=dict(max_pages=(1 << 26) + 1, ld_table=1 << 27))),
    (OK, dict(rows=dict(B=0))),
])
def test_shared_refusals(lib, call, want, kw):
    assert call(lib, **kw) == want


def test_rotary_refusals(lib):
    assert _rotary(lib, R=63) == INV and _rotary(lib, R=-2) == INV and _rotary(lib, R=66) == INV
    assert _rotary(lib, inv=None) == INV
    assert _rotary(lib, mag=float("nan")) == INV
    assert _rotary(lib, k=dict(p=None)) == INV and _rotary(lib, v=dict(p=None)) == INV
    assert _rotary(lib, q=dict(p=FAKE + 1)) == UNS


def test_attention_refusals(lib):
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _attend(lib, scale=s) == INV
    assert _attend(lib, window=-1) == INV
    assert _attend(lib, Hq=7) == INV             # not a multiple of the cache's heads
    for D in (8, 20, 136):
        assert _attend(lib, D=D) == UNS
    for ps in (4, 12, 24, 2048):
        assert _attend(lib, ps=ps) == UNS
    assert _attend(lib, q=dict(p=FAKE + 2)) == UNS
    assert _attend(lib, out=dict(token_stride=8 * 64 + 4)) == UNS
    assert _attend(lib, cache=dict(v=FAKE + 8)) == UNS
    assert _attend(lib, cache=dict(k_page_stride=16 * 128 + 4)) == UNS
    assert _attend(lib, lse=FAKE + 2) == UNS
    assert _attend(lib, ws=None) == WS and _attend(lib, ws=FAKE + 16) == WS
    need = lib.dspark_block_attention_workspace_bytes(8, 8, 2, 64)
    assert need > 0 and _attend(lib, wsb=need - 1) == WS


def test_workspace_bytes(lib):
    f = lib.dspark_block_attention_workspace_bytes
    assert f(8, 32, 8, 128) > 0 and f(0, 32, 8, 128) >= 0
    assert f(8, 32, 8, 144) == 0 and f(8, 32, 8, 12) == 0 and f(8, 30, 8, 128) == 0
    assert f(-1, 32, 8, 128) == 0 and f(8, 0, 8, 128) == 0
    assert f(1, 32, 8, 128) <= f(8, 32, 8, 128) <= f(4096, 32, 8, 128) < 64 << 20


def _tensors(dev="cpu", **over):
    bf, i32 = dict(dtype=torch.bfloat16, device=dev), dict(dtype=torch.int32, device=dev)
    t = dict(q=torch.zeros(2, 3, 4, 64, **bf), k=torch.zeros(2, 3, 2, 64, **bf),
             v=torch.zeros(2, 3, 2, 64, **bf), k_pages=torch.zeros(5, 16, 2, 64, **bf),
             v_pages=torch.zeros(5, 16, 2, 64, **bf), page_table=torch.zeros(2, 2, **i32),
             kv_len=torch.full((2,), 3, **i32),
             inv_freq=torch.ones(32, dtype=torch.float32, device=dev))
    t.update(over)
    return t


def test_wrappers_need_cuda():
    t = _tensors()
    with pytest.raises(RuntimeError):
        dv.rotary_append(**t)
    for key in ("k", "v", "inv_freq"):
        t.pop(key)
    with pytest.raises(RuntimeError):
        dv.block_attention(**t)


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(2, 3, 4, 32, dtype=torch.bfloat16)),
    dict(k_pages=torch.zeros(5, 16, 2, 64, dtype=torch.float16)),
    dict(v_pages=torch.zeros(5, 8, 2, 64, dtype=torch.bfloat16)),
    dict(k_pages=torch.zeros(5, 16, 64, 2, dtype=torch.bfloat16).transpose(2, 3)),
    dict(page_table=torch.zeros(2, 2, dtype=torch.int64)),
    dict(page_table=torch.zeros(3, 2, dtype=torch.int32)),
    dict(page_table=torch.zeros(2, 4, dtype=torch.int32)[:, ::2]),
])
def test_cache_layout_checks(over):
    t = _tensors(**over)
    with pytest.raises(ValueError):
        ch._check_cache(t["k_pages"], t["v_pages"], t["page_table"], t["kv_len"],
                        t["q"].shape[-1], t["q"].dtype, -1)


def test_head_layout_checks():
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    shape = torch.Size((2, 3, 2, 64))
    wide = torch.zeros(2, 3, 6, 64, dtype=torch.bfloat16)
    ok = ch._heads(wide[:, :, :2], shape, q.dtype, -1, "k")
    assert (ok.seq_stride, ok.token_stride, ok.head_stride) == (3 * 6 * 64, 6 * 64, 64)
    for bad in (torch.zeros(2, 3, 2, 64), torch.zeros(2, 3, 3, 64, dtype=torch.bfloat16),
                torch.zeros(2, 4, 2, 64, dtype=torch.bfloat16),
                torch.zeros(6, 2, 64, dtype=torch.bfloat16),
                torch.zeros(2, 3, 64, 2, dtype=torch.bfloat16).transpose(2, 3)):
        with pytest.raises(ValueError):
            ch._heads(bad, shape, q.dtype, -1, "k")


def test_struct_sizes_match_the_header():
    """The ctypes layouts are those of a 64-bit C compiler for the header's structs."""
    assert ctypes.sizeof(ch.Heads) == 32 and ctypes.sizeof(ch.Rows) == 24
    assert ctypes.sizeof(ch.KvCache) == 8 * 8 + 4 * 4 + 8 + 8 + 8 + 8

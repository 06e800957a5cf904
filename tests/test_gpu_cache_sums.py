"""block_attention's sums over long items: the tensor cores cut products off below the sum that
they join, so a sum over many tiles must not stay with them."""

import pytest
import torch

import lossless_draft_verification_speculative_b200 as dv
from cache_helpers import DEV, DT, HALF_STEP

pytestmark = pytest.mark.gpu

# 128 products a tile, each cut off 25 places below the sum, over the tiles that a sum stays; and
# eight results of 24 places a tile
CUT = {d: t * (128 * 2.0 ** -25 + 8 * 2.0 ** -24) for d, t in (("f16", 64), ("bf16", 256))}


def _pool(pages, ps, Hk, D, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    k = torch.randn(pages, ps, Hk, D, generator=g, device=DEV)
    v = 0.5 + torch.rand(pages, ps, Hk, D, generator=g, device=DEV)
    return k.to(DT[dtype]), v.to(DT[dtype]), g


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,tiles", [(256, 64), (256, 65), (256, 1000), (64, 129), (64, 2048),
                                     (256, 257), (64, 513)])
def test_equal_weights_over_many_tiles(dtype, D, n, tiles):
    """Keys of zeros: a row is the mean of its values. One item per CTA, of 256 rows or of 64 (whose
    tiles two groups share)."""
    Hk, ps = 148, 128
    k, v, _ = _pool(8, ps, Hk, D, dtype, 1)
    table = (torch.arange(tiles, device=DEV) % 8).to(torch.int32)[None]
    L = torch.tensor([tiles * ps], dtype=torch.int32, device=DEV)
    q = torch.ones(1, n, Hk, D, dtype=DT[dtype], device=DEV)
    out = dv.block_attention(q, torch.zeros_like(k), v, table, L, causal=False)[0].double()
    times = torch.bincount(table[0].long(), minlength=8).double()
    want = (v.double().sum(1) * times[:, None, None]).sum(0) / (tiles * ps)   # [Hk, D]
    rel = (out - want) / want
    u = HALF_STEP[dtype]
    assert rel.abs().max() <= u + CUT[dtype]
    # n rows alike: Hk D results, each rounded either way
    assert rel.mean().abs() <= CUT[dtype] / 2 + 4 * u / (Hk * D) ** 0.5


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,D,tiles", [(130, 128, 700), (256, 64, 3000), (40, 64, 1500)])
def test_moving_maxima_over_many_tiles(dtype, n, D, tiles):
    """Random keys, with larger ones a third of the way and at the end, so that the maximum moves
    after sums have left tensor memory."""
    Hk, ps = 148, 128
    k, v, g = _pool(10, ps, Hk, D, dtype, 2)
    table = torch.arange(tiles, device=DEV) % 8
    table[tiles // 3], table[-1] = 8, 9
    q = torch.randn(1, n, Hk, D, generator=g, device=DEV).to(DT[dtype])
    lift = q[0].float().mean(0) * (D / q[0].float().mean(0).pow(2).sum(-1, keepdim=True)) * 0.5
    k[8, 5:40] = (k[8, 5:40].float() + lift).to(DT[dtype])
    k[9, 77] = (k[9, 77].float() + 2 * lift).to(DT[dtype])
    L = torch.tensor([tiles * ps], dtype=torch.int32, device=DEV)
    lse = torch.zeros(1, n, Hk, device=DEV)
    out = dv.block_attention(q, k, v, table.to(torch.int32)[None], L, causal=False, lse=lse)
    times = torch.bincount(table, minlength=10).double().repeat_interleave(ps)
    u, errs = HALF_STEP[dtype], []
    for h in range(Hk):
        K, V = k[:, :, h].reshape(-1, D).double(), v[:, :, h].reshape(-1, D).double()
        z = q[0, :, h].double() @ K.T * D ** -0.5 + times.log()
        want_lse = z.logsumexp(-1)
        w = (z - want_lse[:, None]).exp()
        want = w @ V
        qk = (q[0, :, h].double().abs() @ K.abs().T).amax(-1) * D ** -0.5
        e = 2 * (qk * (D + 4) * 2.0 ** -24 + 2.0 ** -21)  # of a weight, from its float32 score
        err = (out[0, :, h].double() - want) / want
        assert (err.abs() <= (2 * u + CUT[dtype] + e[:, None]) * 1.01).all(), h
        # l: a tile's sum of 128 is added in float32, tiles times
        assert ((lse[0, :, h].double() - want_lse).abs() <=
                e + (tiles + 128) * 2.0 ** -24 + 2.0 ** -22 * want_lse.abs() + 2.0 ** -22).all(), h
        errs.append((err.mean().abs() - e.max()).item())
    # roundings to the nearest go either way; the cut-off is a bias (each row has a thousand weights
    # of its own, each head its own values)
    assert max(errs) <= CUT[dtype] + 4 * u / D ** 0.5, max(errs)


def test_a_sum_of_201326592_ones():
    """256 rows of each of 148 heads over 201326592 positions with equal weights: the sums of ones
    and twos are exact in float32 (256 tiles at a time, then 32768 at a time)."""
    L, ps, Hk, n, D = 3 << 26, 1024, 148, 256, 16
    pages = torch.zeros(2, 1, ps, Hk, D, dtype=torch.bfloat16, device=DEV)
    pages[1, ..., :8], pages[1, ..., 8:] = 1.0, 2.0
    table = torch.zeros(1, L // ps, dtype=torch.int32, device=DEV)
    q = torch.ones(1, n, Hk, D, dtype=torch.bfloat16, device=DEV)
    out = dv.block_attention(q, pages[0], pages[1], table,
                             torch.tensor([L], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert (out[..., :8] == 1.0).all() and (out[..., 8:] == 2.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [4, 256])
@pytest.mark.parametrize("tiles", [148 * 300, 148 * 700 + 77])
def test_long_pieces_are_summed_and_joined(dtype, n, tiles):
    """One cache head over millions of positions: every CTA has a piece of hundreds of tiles, whose
    sums leave tensor memory before the pieces are joined; every page but two is of eight."""
    ps, D = 128, 64
    k, v, g = _pool(10, ps, 1, D, dtype, 3)
    table = torch.arange(tiles, device=DEV) % 8
    table[tiles // 3], table[-1] = 8, 9
    k[8] *= 2
    q = torch.randn(1, n, 1, D, generator=g, device=DEV).to(DT[dtype])
    lse = torch.zeros(1, n, 1, device=DEV)
    out = dv.block_attention(q, k, v, table.to(torch.int32)[None],
                             torch.tensor([tiles * ps], dtype=torch.int32, device=DEV),
                             causal=False, lse=lse)
    times = torch.bincount(table, minlength=10).double().repeat_interleave(ps)
    K, V = k.reshape(-1, D).double(), v.reshape(-1, D).double()
    z = q[0, :, 0].double() @ K.T * D ** -0.5 + times.log()
    want_lse = z.logsumexp(-1)
    want = (z - want_lse[:, None]).exp() @ V
    e = 2 * ((q[0, :, 0].double().abs() @ K.abs().T).amax(-1) * D ** -0.5 * (D + 4) * 2.0 ** -24
             + 2.0 ** -21)
    err = (out[0, :, 0].double() - want).abs() / want
    assert (err <= (2 * HALF_STEP[dtype] + CUT[dtype] + e[:, None]) * 1.01).all()
    per = tiles // 148 + 128 + 148  # additions: a piece's tiles, a tile's places, the pieces
    assert ((lse[0, :, 0].double() - want_lse).abs() <=
            e + per * 2.0 ** -24 + 2.0 ** -22 * want_lse.abs() + 2.0 ** -22).all()

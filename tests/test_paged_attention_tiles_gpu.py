"""The kernel of many rows over the paged cache: page sizes and layouts, pages that
are missing, masks and values that are not finite, for all of its head sizes."""
import math

import pytest
import torch

from paged import BF, DEV, E4M3, F16, Batch, attend, check, queries

pytestmark = pytest.mark.gpu

KINDS = [(BF, BF), (F16, F16), (BF, E4M3), (F16, E4M3)]


def run(b, q, **kw):
    assert b.max_rows * (q.shape[1] // b.heads) > 16, "few rows take another kernel"
    check(b, q, attend(b, q, b.heads, **kw), **kw)


# boxes of tiled loads hold the largest power of two that divides a page, from 8 slots up to a tile;
# other pages are copied in pieces of 16 bytes
@pytest.mark.parametrize("page", [1, 2, 4, 7, 8, 16, 24, 40, 64, 100, 128, 200, 256, 1000])
@pytest.mark.parametrize("layout,q_type,cache", [
    ("head", BF, BF), ("slot", BF, BF), ("wide", BF, BF), ("slot", F16, F16), ("head", BF, E4M3), ("slot", F16, E4M3), ("wide", BF, E4M3)])
@pytest.mark.parametrize("dim", [64, 80, 128, 256])
def test_pages_and_layouts(page, layout, q_type, cache, dim):
    b = Batch([(40, 401), (1, 128), (30, 65), (0, 9), (5, 3)], 2, dim, page, cache, layout=layout, wide=2)
    run(b, queries(b, 8, q_type))


@pytest.mark.parametrize("dim", [16, 128, 144, 192, 256])
@pytest.mark.parametrize("q_type,cache", KINDS)
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 100), (True, 333), (False, 0), (False, 1), (False, 64), (False, 200)])
def test_masks(dim, q_type, cache, causal, window):
    b = Batch([(300, 433), (70, 100), (1, 1), (0, 50), (20, 8), (140, 700)], 1, dim, 32, cache, first=3, behind=2)
    run(b, queries(b, 2, q_type), causal=causal, window=window)


def seen_pages(b, q, got, gone, causal, window):
    """As check(), the positions in gone[s] being seen by no token."""
    half = torch.finfo(q.dtype).eps / 2
    group = q.shape[1] // b.heads
    for s, (rows, length) in enumerate(b.seqs):
        at = slice(b.used[s], b.used[s] + rows)
        k, v = (x.repeat_interleave(group, dim=1) for x in b.held[s])
        pos, mine = torch.arange(length, device=DEV), torch.arange(length - rows, length, device=DEV)[:, None]
        sees = ~gone[s] & ((pos <= mine) if causal else torch.ones_like(pos <= mine))
        if window:
            sees = sees & (pos > mine - window)
        hide = ~sees[:, None, :]
        z = torch.einsum("thd,lhd->thl", q[at].double(), k) * b.dim ** -0.5
        size = (torch.einsum("thd,lhd->thl", q[at].double().abs(), k.abs()) * b.dim ** -0.5).masked_fill(hide, 0.0).amax(-1)
        z = z.masked_fill(hide, -math.inf)
        m = z.amax(-1, keepdim=True)
        p = torch.exp(z - torch.where(m > -math.inf, m, torch.zeros_like(m)))
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, torch.zeros_like(p))
        want, lse = torch.einsum("thl,lhd->thd", p, v), (m + torch.log(total))[..., 0]
        dz = size * ((b.dim + 4) * 2.0 ** -23 + 2.0 ** -21) + length * 2.0 ** -23 + 2.0 ** -20
        d = half * want.abs() + torch.einsum("thl,lhd->thd", p, v.abs()) * (half + 2 * dz[..., None]) * (1 + half) + 2.0 ** -24
        far = (got[0][at].double() - want).abs() - d
        assert (far <= 0).all(), f"out: {far.max().item()} over its bound"
        none = torch.isneginf(lse)
        assert torch.isneginf(got[1][at][none]).all() and (got[0][at][none] == 0).all()
        assert ((got[1][at].double() - lse).abs() <= dz + 2.0 ** -22 * lse.abs())[~none].all()


@pytest.mark.parametrize("q_type,cache", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 24, 128, 20])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 190)])
@pytest.mark.parametrize("rows,few", [(150, False), (70, False), (2, True)])
def test_missing_pages(q_type, cache, dim, page, causal, window, rows, few):
    """In a first, a middle and the last tile, in either half of one, a whole tile and more,
    and a sequence's only ones, with bad entries of each kind."""
    b = Batch([(rows, 900), (rows, 700), (rows, 300), (rows, 512), (rows, 100)], 2, dim, page, cache, max_rows=rows)
    assert few == (rows * 2 <= 16)
    q = queries(b, 4, q_type)
    lost = [[(400, 420), (600, 601)], [(0, 1), (699, 700)], [(64, 300)], [(129, 150), (200, 201), (256, 400)], [(0, 100)]]
    bad, gone = [-1, b.n_pages, 0x7FFFFFFF, -(1 << 31)], []
    for s, (_, length) in enumerate(b.seqs):
        pages = sorted({p // page for lo, hi in lost[s] for p in range(lo, hi)})
        for i, p in enumerate(pages):
            b.table[s, p] = bad[(s + i) % 4]
        gone.append(torch.isin(torch.arange(length, device=DEV) // page, torch.tensor(pages, device=DEV)))
    seen_pages(b, q, attend(b, q, 2, causal=causal, window=window), gone, causal, window)


@pytest.mark.parametrize("q_type,cache", KINDS)
@pytest.mark.parametrize("dim", [128, 192, 256])
@pytest.mark.parametrize("rows,window", [(40, 0), (200, 0), (200, 100)])
def test_what_a_row_does_not_see_may_be_anything(q_type, cache, dim, rows, window):
    """Keys and values of one position that are not finite change the rows that see
    it, and no others' lse."""
    seqs = [(rows, 460), (3, 200)]
    b = Batch(seqs, 2, dim, 16, cache)
    q = queries(b, 4, q_type)
    clean, clean_lse = attend(b, q, 2, window=window)
    check(b, q, (clean, clean_lse), window=window)
    for which in "kv":
        for place in (459, 460 - rows // 2 - 1, 130):
            b = Batch(seqs, 2, dim, 16, cache)
            page, slot = b.table[0, place // 16].item(), place % 16
            if cache == E4M3:
                getattr(b, which).view(torch.uint8)[page, slot, 1] = 0x7F
            else:
                getattr(b, which)[page, slot, 1] = math.inf if place == 130 else math.nan
            out, lse = attend(b, q, 2, window=window)
            mine = torch.arange(460 - rows, 460, device=DEV)
            odd = torch.zeros(len(q), 4, dtype=torch.bool, device=DEV)
            odd[:rows, 2:] = ((mine >= place) & ((mine - place < window) if window else True))[:, None]
            assert torch.isfinite(out[~odd]).all() and torch.equal(lse[~odd], clean_lse[~odd])
            # rows may be taken again one position at a time: the same exponentials' products in another order
            d = (out.float() - clean.float()).abs()[~odd]
            assert (d <= 2.0 ** -6 * (1 + clean.float().abs()[~odd])).all()
            if which == "v":
                assert not torch.isfinite(out[odd]).any() and torch.equal(lse, clean_lse)
            elif place != 130:
                assert torch.isnan(lse[odd]).all()


@pytest.mark.parametrize("q_type,cache", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("length", [460, 20000])
def test_a_key_that_is_seen_beside_a_value_that_is_not(q_type, cache, dim, length):
    """Rows that see a NaN key are NaN, also where a value behind them has their rows
    taken again; the rows before it are not."""
    rows = 200
    b = Batch([(rows, length)], 1, dim, 16, cache)
    q = queries(b, 2, q_type)
    clean = attend(b, q, 1)
    check(b, q, clean)
    key, value = length - 100, length - 10
    for name, pos in (("k", key), ("v", value)):
        page, slot = b.table[0, pos // 16].item(), pos % 16
        if cache == E4M3:
            getattr(b, name).view(torch.uint8)[page, slot, 0] = 0x7F
        else:
            getattr(b, name)[page, slot, 0] = math.nan
    out, lse = attend(b, q, 1)
    sees = torch.arange(length - rows, length, device=DEV) >= key
    assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all()
    assert torch.equal(lse[~sees], clean[1][~sees])
    d = (out.float() - clean[0].float()).abs()[~sees]
    assert (d <= 2.0 ** -6 * (1 + clean[0].float().abs()[~sees])).all()

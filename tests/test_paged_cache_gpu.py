"""Writing rows into the paged cache and reading them back, against 64 bits."""
import math

import pytest
import torch

from paged import BF, DEV, E4M3, F16, F32, Batch, quantised
from quantized_routed_expert_gemv_gb300.device import PagedCache, Sequences

pytestmark = pytest.mark.gpu


def rows_of(b, dtype, pad=0, seed=3, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(b.rows, b.heads * b.dim + pad, dtype=dtype, device=DEV)[:, :b.heads * b.dim]
    x = x.unflatten(1, (b.heads, b.dim))
    x.copy_(torch.randn(b.rows, b.heads, b.dim, generator=g, device=DEV) * size)
    return x


def raw(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t.view(torch.int16) if t.dtype in (BF, F16) else t.view(torch.int32)


def expect_written(b, k, v, before):
    """The cache that writing should leave."""
    want = {n: raw(t).clone() for n, t in before.items()}
    for s, (rows, length) in enumerate(b.seqs):
        skip = max(0, rows - length)
        pos = torch.arange(length - rows + skip, length, device=DEV)
        page, slot = b.slots(s, pos)
        for name, x in (("k", k), ("v", v)):
            x = x[b.used[s] + skip:b.used[s] + rows]
            if b.type == E4M3:
                codes, scale = quantised(x)
                want[name][page, slot] = raw(codes.float().to(E4M3))
                want[name + "_scale"][page, slot] = raw(scale.float())
            else:
                want[name][page, slot] = raw(x.float().to(b.type))
    return want


def state(b):
    names = ("k", "v") + (("k_scale", "v_scale") if b.type == E4M3 else ())
    return {n: getattr(b, n) for n in names}


SEQS = [[(1, 1)], [(5, 9), (0, 4), (1, 30), (7, 3), (12, 12)], [(1, 40)] * 70, [(0, 0), (0, 5), (3, 100)]]


@pytest.mark.parametrize("cache,src", [(E4M3, BF), (E4M3, F32), (E4M3, F16), (BF, BF), (BF, F32), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("seqs,heads,dim,page,pad,layout", [
    (0, 1, 16, 1, 0, "head"), (0, 8, 128, 16, 0, "slot"), (1, 3, 80, 7, 0, "head"), (1, 4, 64, 16, 3, "slot"),
    (2, 2, 256, 24, 8, "wide"), (3, 5, 48, 64, 1, "wide"), (2, 1, 112, 5, 0, "slot")])
def test_write(cache, src, seqs, heads, dim, page, pad, layout):
    b = Batch(SEQS[seqs], heads, dim, page, cache, first=seqs % 2 * 2, behind=seqs, layout=layout, wide=seqs)
    k, v = rows_of(b, src, pad), rows_of(b, src, pad, seed=4, size=30.0)
    k[:1, :1] = 0.0
    before = {n: t.clone() for n, t in state(b).items()}
    b.cache().write(k, v, b.sequences())
    torch.cuda.synchronize()
    want = expect_written(b, k, v, before)
    for n, t in state(b).items():
        assert torch.equal(raw(t), want[n]), n


@pytest.mark.parametrize("top", [448.0, 448.0 * 2.0 ** -9, 449.0, 447.9, 480.0, 2.0 ** -149, 2.0 ** -118, 3.0e38, 1.0, 65504.0])
def test_scales_at_powers_of_two(top):
    """Largest magnitudes on and beside a scale's border, and the ends of fp32."""
    b = Batch([(6, 6)], 2, 32, 4, E4M3)
    k = rows_of(b, F32).clamp(-1, 1) * top * 0.5
    k[:, :, 5] = -top
    before = {n: t.clone() for n, t in state(b).items()}
    b.cache().write(k, k, b.sequences())
    torch.cuda.synchronize()
    want = expect_written(b, k, k, before)
    for n, t in state(b).items():
        assert torch.equal(raw(t), want[n]), n


def test_ties_go_to_even():
    b = Batch([(1, 1)], 1, 16, 1, E4M3)
    # halfway between neighbours of e4m3 at scale 1: 17 -> 16, 19 -> 20, subnormal 0.5 and 1.5 of 2^-9
    x = torch.tensor([448.0, 17, 19, 21, 23, 2.0 ** -10, 1.5 * 2.0 ** -9, -17, -19, 0.0, 1, 240, 232, 2.0 ** -6, 9.5, 8.5],
                     device=DEV)
    b.cache().write(x.view(1, 1, 16), x.view(1, 1, 16), b.sequences())
    got = b.k[b.table[0, 0].item(), 0, 0].float()
    torch.cuda.synchronize()
    want = [448, 16, 20, 20, 24, 0, 2.0 ** -8, -16, -20, 0, 1, 240, 224, 2.0 ** -6, 10, 8]
    assert got.tolist()[:11] + got.tolist()[13:] == want[:11] + want[13:]
    assert got[11] == 240 and got[12] in (224, 240)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_head_that_is_not_finite(bad):
    b = Batch([(3, 3)], 2, 64, 16, E4M3)
    k, v = rows_of(b, BF), rows_of(b, BF, seed=5)
    k[1, 0, 17], v[2, 1, 3] = bad, bad
    cache = b.cache()
    cache.write(k, v, b.sequences())
    ko, vo = cache.read(b.sequences(), rows=3, out_type=F32)
    torch.cuda.synchronize()
    nan_k, nan_v = torch.isnan(ko).all(-1), torch.isnan(vo).all(-1)
    assert nan_k.nonzero().tolist() == [[1, 0]] and nan_v.nonzero().tolist() == [[2, 1]]
    assert torch.isnan(ko).any(-1).equal(nan_k) and torch.isnan(vo).any(-1).equal(nan_v)


@pytest.mark.parametrize("cache,dst", [(E4M3, BF), (E4M3, F32), (E4M3, F16), (BF, F32), (F16, BF), (BF, BF)])
@pytest.mark.parametrize("seqs,heads,dim,page,pad,layout", [
    (0, 2, 32, 3, 0, "slot"), (1, 3, 80, 7, 5, "head"), (2, 8, 128, 16, 0, "wide"), (3, 1, 256, 16, 8, "head")])
def test_read(cache, dst, seqs, heads, dim, page, pad, layout):
    b = Batch(SEQS[seqs], heads, dim, page, cache, first=1, behind=2, layout=layout)
    ko, vo = rows_of(b, dst, pad), rows_of(b, dst, pad)
    ko.fill_(7.0), vo.fill_(7.0)
    b.cache().read(b.sequences(), k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    for i, got in enumerate((ko, vo)):
        want = torch.full_like(got, 7.0)
        for s, (rows, length) in enumerate(b.seqs):
            skip = max(0, rows - length)
            want[b.used[s]:b.used[s] + skip] = 0.0
            want[b.used[s] + skip:b.used[s] + rows] = b.held[s][i][length - rows + skip:].float().to(dst)
        assert torch.equal(got, want)


def test_missing_pages_and_sizes_outside_the_contract():
    """Pages that do not exist are neither written nor read, lengths beyond the
    table are cut, and starts beyond the rows too."""
    b = Batch([(8, 8), (8, 8), (8, 8)], 2, 64, 2, BF)
    b.table[0, 1], b.table[1, 2], b.table[2, 0] = -1, b.n_pages, 0x7FFFFFFF
    before = {n: t.clone() for n, t in state(b).items()}
    k, v = rows_of(b, BF), rows_of(b, BF, seed=6)
    cache = b.cache()
    cache.write(k, v, b.sequences())
    ko, vo = cache.read(b.sequences(), rows=24)
    torch.cuda.synchronize()
    lost = [2, 3, 12, 13, 16, 17]
    kept = [r for r in range(24) if r not in lost]
    assert (ko[lost] == 0).all() and (vo[lost] == 0).all()
    assert torch.equal(ko[kept], k[kept]) and torch.equal(vo[kept], v[kept])
    pages = b.table.flatten().tolist()
    others = [p for p in range(b.n_pages) if p not in pages]
    assert torch.equal(raw(b.k)[others], raw(before["k"])[others])
    # a length beyond the table counts as the table's end, negative ones as 0, starts as cut to the rows
    b2 = Batch([(4, 8), (4, 8), (4, 8)], 1, 16, 4, BF)
    b2.kv_lens.copy_(torch.tensor([1 << 30, -5, 8]))
    b2.starts.copy_(torch.tensor([0, 4, 8, 1 << 30]))
    ko, _ = b2.cache().read(b2.sequences(), rows=12)
    torch.cuda.synchronize()
    assert torch.equal(ko[:4], b2.held[0][0][4:].to(BF)) and (ko[4:8] == 0).all()
    assert torch.equal(ko[8:], b2.held[2][0][4:].to(BF))


def test_places_beyond_32_bits():
    """Pages whose elements lie beyond 2^32 bytes and 2^31 elements."""
    n_pages = (1 << 32) // (16 * 8 * 128) + 40
    cache = PagedCache.empty(n_pages, 16, 8, 128, E4M3)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2]], dtype=torch.int32, device=DEV)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    seqs = Sequences(i32(0, 48), i32(48), table)
    k, v = torch.randn(48, 8, 128, device=DEV), torch.randn(48, 8, 128, device=DEV)
    cache.write(k, v, seqs)
    ko, vo = cache.read(seqs, rows=48, out_type=F32)
    torch.cuda.synchronize()
    for x, got in ((k, ko), (v, vo)):
        codes, scale = quantised(x)
        assert torch.equal(got.double(), codes * scale[..., None])


def test_captured_and_replayed():
    """A graph follows the tensors' contents: rows, sequences and pages."""
    b = Batch([(2, 30), (3, 20)], 2, 64, 4, E4M3, behind=4)
    k, v = rows_of(b, BF), rows_of(b, BF, seed=7)
    cache, seqs = b.cache(), b.sequences()
    ko, vo = (torch.zeros(b.rows, 2, 64, dtype=BF, device=DEV) for _ in range(2))
    cache.write(k, v, seqs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.write(k, v, seqs)
        cache.read(seqs, k_out=ko, v_out=vo)
    for rows, lens, seed in (((2, 3), (30, 20), 8), ((1, 5), (7, 18), 9), ((4, 5), (28, 5), 10)):
        k.copy_(rows_of(b, BF, seed=seed))
        b.starts.copy_(torch.tensor([0, rows[0], sum(rows)]))
        b.kv_lens.copy_(torch.tensor(lens))
        ko.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        codes, scale = quantised(k)
        want = (codes * scale[..., None]).to(BF)
        assert torch.equal(ko[:sum(rows)], want[:sum(rows)]) and (ko[sum(rows):] == 7.0).all()


def test_no_rows_and_no_sequences():
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    cache = PagedCache.empty(4, 16, 2, 64, BF)
    none = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    cache.write(none, none, Sequences(i32(0, 0), i32(0), i32(0).view(1, 1)))
    cache.write(none, none, Sequences(i32(0), torch.empty(0, dtype=torch.int32, device=DEV),
                                      torch.empty(0, 3, dtype=torch.int32, device=DEV)))
    some = torch.ones(3, 2, 64, dtype=BF, device=DEV)
    empty = PagedCache.empty(0, 16, 2, 64, BF)
    empty.write(some, some, Sequences(i32(0, 3), i32(3), i32(0).view(1, 1)))
    k, _ = empty.read(Sequences(i32(0, 3), i32(3), i32(0).view(1, 1)), rows=3)
    torch.cuda.synchronize()
    assert (k == 0).all()

"""Attention of new tokens over the paged cache, against 64 bits."""
import math

import pytest
import torch

from paged import BF, DEV, E4M3, F16, F32, Batch, attend, check, queries, reference
from quantized_routed_expert_gemv_gb300.device import PagedAttention, PagedCache, Sequences

pytestmark = pytest.mark.gpu

KINDS = [(BF, BF), (F16, F16), (BF, E4M3), (F16, E4M3)]


def run(b, q, **kw):
    check(b, q, attend(b, q, b.heads, **kw), **kw)


@pytest.mark.parametrize("q_type,cache", KINDS)
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("rows", [1, 5])
def test_types_and_head_sizes(q_type, cache, dim, rows):
    b = Batch([(rows, 150), (rows, rows), (rows, 700)], 2, dim, 16, cache)
    run(b, queries(b, 8, q_type))


@pytest.mark.parametrize("kv_heads,group", [(1, 1), (3, 1), (2, 3), (1, 8), (2, 16), (2, 17), (1, 20), (1, 128)])
@pytest.mark.parametrize("rows", [1, 2, 37])
def test_head_layouts(kv_heads, group, rows):
    b = Batch([(rows, 300), (1, 1), (rows, 64)], kv_heads, 64, 16)
    run(b, queries(b, kv_heads * group, BF))


@pytest.mark.parametrize("page", [1, 2, 7, 16, 24, 64, 100, 128, 200, 1000])
@pytest.mark.parametrize("layout,cache", [("head", BF), ("slot", E4M3), ("wide", BF), ("wide", E4M3)])
def test_pages(page, layout, cache):
    b = Batch([(3, 401), (1, 128), (2, 65)], 2, 64, page, cache, layout=layout, wide=2)
    run(b, queries(b, 8, BF))


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 20011])
@pytest.mark.parametrize("rows", [1, 3])
def test_lengths(length, rows):
    """Rows before the first position see nothing."""
    b = Batch([(rows, length)], 2, 128, 16)
    run(b, queries(b, 16, BF))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 2, 17, 64, 128, 1000, 0x7FFFFFFF])
@pytest.mark.parametrize("rows", [1, 70, 300])
def test_masks(causal, window, rows):
    b = Batch([(rows, 333), (rows, 100), (1, 1), (0, 50)], 1, 64, 32, first=3, behind=2)
    run(b, queries(b, 4, BF), causal=causal, window=window)


@pytest.mark.parametrize("q_type,cache", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_chunks(q_type, cache, dim):
    """Many rows: chunks behind a prefix, prompts of their own, single tokens, a
    sequence without rows, one with more rows than positions."""
    b = Batch([(260, 600), (130, 130), (1, 900), (0, 77), (90, 40), (1, 1)], 2, dim, 16, cache, behind=5)
    run(b, queries(b, 10, q_type))


@pytest.mark.parametrize("n", [33, 129, 300, 1111])
def test_many_sequences(n):
    g = torch.Generator().manual_seed(n)
    seqs = [(int(torch.randint(0, 3, (), generator=g)), int(torch.randint(0, 90, (), generator=g))) for _ in range(n)]
    b = Batch(seqs, 2, 64, 16)
    run(b, queries(b, 4, BF))


@pytest.mark.parametrize("n", [500, 513, 1100])
def test_many_sequences_in_large_tiles(n):
    """The hint takes the kernel of many rows, which looks at 512 sequences at a time."""
    g = torch.Generator().manual_seed(n)
    seqs = [(int(torch.randint(0, 4, (), generator=g)), int(torch.randint(0, 150, (), generator=g))) for _ in range(n)]
    b = Batch(seqs, 2, 64, 16, max_rows=1000)
    run(b, queries(b, 4, BF))


@pytest.mark.parametrize("max_rows", [1, 1000])
@pytest.mark.parametrize("q_type,powers", [(BF, (-120, -40, 0, 6, 9, 60)), (F16, (-14, -3, 0, 4, 5))])
def test_scales_far_from_one(max_rows, q_type, powers):
    """Heads of an e4m3 cache whose magnitudes differ by powers of two, keys and
    values alike, and queries that bring z back to about one."""
    b = Batch([(3, 300), (2, 40)], 1, 64, 16, E4M3, max_rows=max_rows)
    g = torch.Generator(device=DEV).manual_seed(3)
    for kp in powers[:2] + powers[-2:]:
        for s, (_, length) in enumerate(b.seqs):
            pos = torch.arange(length, device=DEV)
            pick = torch.tensor(powers, device=DEV, dtype=torch.float64)[torch.randint(0, len(powers), (length, 1, 1), generator=g, device=DEV)]
            k, v = (torch.randn(length, 1, 64, generator=g, device=DEV).double().clamp(-3, 3) for _ in range(2))
            b.held[s] = [b.put(s, "k", pos, k * 2.0 ** kp), b.put(s, "v", pos, v * torch.exp2(pick))]
        q = queries(b, 4, q_type)
        run(b, q, scale=0.125 * 2.0 ** -kp)


@pytest.mark.parametrize("max_rows", [1, 1000])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** 90])
def test_queries_far_from_one(max_rows, size):
    """bfloat16 queries beyond float16's range over an e4m3 cache; a row of
    zeros, and rows whose elements differ by many powers of two."""
    b = Batch([(3, 200), (1, 77)], 2, 80, 16, E4M3, max_rows=max_rows)
    q = queries(b, 8, BF, size=size)
    q[1, 3] = 0.0
    q[0, 2] *= torch.exp2(-torch.arange(80, device=DEV) // 4.0).to(BF)
    run(b, q, scale=0.1 / size)


@pytest.mark.parametrize("seqs,heads,group", [
    ([(1, 50000)], 1, 8), ([(1, 30000), (1, 10), (1, 7000)], 2, 4), ([(2, 9000)] * 3, 4, 8), ([(40, 6000)], 1, 2)])
def test_keys_split_over_the_gpu(seqs, heads, group):
    """Units that many CTAs share."""
    b = Batch(seqs, heads, 128, 16)
    run(b, queries(b, heads * group, BF))


@pytest.mark.parametrize("q_type,cache", KINDS)
@pytest.mark.parametrize("size,scale", [(8.0, None), (1.0, 3.0), (0.0, None), (1.0, 1e-6)])
def test_sharp_and_flat(q_type, cache, size, scale):
    """Nearly one-hot rows, and uniform ones."""
    b = Batch([(1, 700), (20, 500)], 2, 64, 16, cache)
    run(b, queries(b, 8, q_type, size=size), scale=scale)


@pytest.mark.parametrize("q_type,cache", [(BF, BF), (F16, F16)])
def test_one_position_among_many_small_ones(q_type, cache):
    """One position of weight 1 before 20000 of 2^-24 each, whose values agree:
    small exponentials are not lost to a 16-bit type's range."""
    b = Batch([(1, 20001)], 1, 64, 16, cache)
    k, v = torch.zeros(20001, 1, 64, device=DEV), torch.ones(20001, 1, 64, device=DEV)
    k[0, 0, 0], v[0] = 24 * math.log(2), 0.0
    pos = torch.arange(20001, device=DEV)
    b.held[0] = [b.put(0, "k", pos, k), b.put(0, "v", pos, v)]
    q = torch.zeros(1, 1, 64, dtype=q_type, device=DEV)
    q[0, 0, 0] = 1.0
    run(b, q, scale=1.0)


@pytest.mark.parametrize("cache", [BF, E4M3])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("rows,window,group", [(5, 0, 4), (40, 0, 4), (40, 30, 1), (200, 0, 8), (200, 100, 2), (1, 30, 8)])
def test_what_a_row_does_not_see_may_be_anything(cache, bad, rows, window, group):
    """Keys and values of one position that are not finite change the rows that
    see it, and no other bit of the result."""
    q_type = BF
    b = Batch([(rows, 260)], 2, 64, 16, cache)
    q = queries(b, 2 * group, q_type)
    clean, clean_lse = attend(b, q, 2, window=window)
    check(b, q, (clean, clean_lse), window=window)
    for which in "kv":
        for place in (259, 260 - rows // 2 - 1, max(0, 260 - rows - 20)):
            b2 = Batch([(rows, 260)], 2, 64, 16, cache)
            page, slot = b2.table[0, place // 16].item(), place % 16
            if cache == E4M3:
                getattr(b2, which).view(torch.uint8)[page, slot, 1] = 0x7F
                getattr(b2, which + "_scale")[page, slot, 1] = math.nan
            else:
                getattr(b2, which)[page, slot, 1] = bad
            out, lse = attend(b2, q, 2, window=window)
            mine = torch.arange(260 - rows, 260, device=DEV)
            sees = (mine >= place) & ((mine - place < window) if window else True)
            odd = torch.zeros(rows, 2 * group, dtype=torch.bool, device=DEV)
            odd[:, group:] = sees[:, None]
            d = (out.float() - clean.float()).abs()[~odd]
            assert torch.isfinite(out[~odd]).all() and torch.isfinite(lse[~odd]).all()
            # the same sums, but for tiles that are taken one position at a time
            assert (d <= 2.0 ** -6 * (1 + clean.float().abs()[~odd])).all() and torch.equal(lse[~odd], clean_lse[~odd])
            if which == "v":
                assert not torch.isfinite(out[odd]).any()


def test_keys_of_minus_infinity():
    """z of -inf has no weight; a row of nothing else gives 0 and -inf."""
    b = Batch([(1, 40), (1, 20)], 1, 16, 16)
    q = torch.zeros(2, 2, 16, dtype=BF, device=DEV)
    q[:, :, 0] = 1.0
    for s, pos in ((0, torch.arange(0, 40, 2, device=DEV)), (1, torch.arange(20, device=DEV))):
        page, slot = b.slots(s, pos)
        b.k[page, slot, 0, 0] = -math.inf
    b.held[0] = [x[1::2] for x in b.held[0]]
    b.held[1] = [x[:0] for x in b.held[1]]
    out, lse = attend(b, q, 1, causal=False)
    b.seqs = [(1, 20), (1, 0)]
    check(b, q, (out, lse), causal=False)


def test_missing_pages_are_seen_by_no_token():
    b = Batch([(2, 64), (2, 64), (1, 32)], 2, 64, 16)
    q = queries(b, 4, BF)
    b.table[0, 1], b.table[1, 3], b.table[2, 0], b.table[2, 1] = -1, b.n_pages + 7, -9, 0x7FFFFFFF
    out, lse = attend(b, q, 2, causal=False)
    gone = ((0, slice(16, 32)), (1, slice(48, 64)), (2, slice(0, 32)))
    for s, where in gone:
        keep = torch.ones(b.seqs[s][1], dtype=torch.bool, device=DEV)
        keep[where] = False
        b.held[s] = [x[keep] for x in b.held[s]]
        b.seqs[s] = (b.seqs[s][0], int(keep.sum()))
    check(b, q, (out, lse), causal=False)


@pytest.mark.parametrize("max_rows", [1, 1000])
@pytest.mark.parametrize("cache_type", [BF, E4M3])
def test_a_cache_without_pages(max_rows, cache_type):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    q = torch.ones(5, 4, 64, dtype=BF, device=DEV)
    att, cache = PagedAttention(4, 2, 64), PagedCache.empty(0, 16, 2, 64, cache_type)
    none = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    for table in (i32(0, 1, 2, 3).view(2, 2), none):
        out, lse = torch.full_like(q, 7.0), torch.full((5, 4), 7.0, device=DEV)
        att(q, cache, Sequences(i32(0, 2, 5), i32(20, 3), table, max_rows=max_rows), out=out, lse=lse)
        torch.cuda.synchronize()
        assert (out == 0).all() and torch.isneginf(lse).all() and att.check() == 0


@pytest.mark.parametrize("max_rows", [1, 2, 1000])
@pytest.mark.parametrize("seqs", [[(1, 1)], [(1, 3)] * 5, [(0, 9), (1, 1), (0, 2), (2, 70), (0, 0)], [(1, 1), (1, 400), (0, 5)]])
def test_fewer_tiles_than_ctas(max_rows, seqs):
    """Parts of the work that hold no key tile, at the last sequence's end too;
    the tables and queries end where the last row does."""
    b = Batch(seqs, 2, 64, 16, max_rows=max_rows)
    run(b, queries(b, 4, BF))


def test_sequences_that_share_pages():
    """A common prefix kept once."""
    b = Batch([(1, 100), (3, 90)], 2, 64, 16)
    b.table[1, :4] = b.table[0, :4]
    b.held[1] = [torch.cat((x[:64], y[64:])) for x, y in zip(b.held[0], b.held[1])]
    run(b, queries(b, 8, BF))


def test_queries_and_outputs_inside_wider_rows():
    b = Batch([(3, 90), (20, 50)], 2, 80, 16)
    q = queries(b, 6, BF)
    wide = torch.full((b.rows, 6 * 80 + 24), 9.0, dtype=BF, device=DEV)
    wide[:, 8:488] = q.view(b.rows, -1)
    into = torch.full((b.rows, 6 * 80 + 16), 9.0, dtype=BF, device=DEV)
    att = PagedAttention(6, 2, 80)
    att(wide[:, 8:488].unflatten(1, (6, 80)), b.cache(), b.sequences(), out=into[:, :480].unflatten(1, (6, 80)))
    alone = att(q, b.cache(), b.sequences())
    torch.cuda.synchronize()
    assert torch.equal(into[:, :480], alone.view(b.rows, -1)) and (into[:, 480:] == 9.0).all()


@pytest.mark.parametrize("max_rows", [0, 1, 3, 1000, None])
def test_the_hint_changes_no_result(max_rows):
    """max_rows may be wrong: it chooses a kernel only."""
    b = Batch([(1, 300), (70, 200), (3, 3)], 2, 64, 16, max_rows=max_rows)
    if max_rows is None:
        b.max_rows = None
    run(b, queries(b, 8, BF))


@pytest.mark.parametrize("rows", [1, 150])
def test_the_same_call_gives_the_same_bits(rows):
    b = Batch([(rows, 5000), (rows, 777)], 2, 128, 16)
    q = queries(b, 16, BF)
    first = attend(b, q, 2)
    for _ in range(3):
        out, lse = attend(b, q, 2)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("rows", [1, 60])
def test_captured_and_replayed(rows):
    """Lengths, pages and rows are read at replay; two graphs share a workspace."""
    b = Batch([(rows, 800), (rows, 500)], 2, 64, 16, behind=1)
    q = queries(b, 8, BF)
    att, cache, seqs = PagedAttention(8, 2, 64), b.cache(), b.sequences()
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
    out2 = torch.full_like(q, 7.0)
    att(q, cache, seqs, out=out, lse=lse)
    torch.cuda.synchronize()
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att(q, cache, seqs, out=out, lse=lse)
    with torch.cuda.graph(graph2):
        att(q, cache, seqs, out=out2, causal=False)
    for lens, counts in (((800, 500), (rows, rows)), ((333, 40), (rows, rows)), ((1, 499), (1, rows))):
        b.kv_lens.copy_(torch.tensor(lens))
        b.starts.copy_(torch.tensor([0, counts[0], sum(counts)]))
        q.copy_(queries(b, 8, BF, seed=sum(lens)))
        out.fill_(7.0), lse.fill_(7.0)
        graph.replay(), graph2.replay(), graph.replay()
        torch.cuda.synchronize()
        view = Batch.__new__(Batch)
        view.__dict__.update(b.__dict__)
        view.seqs = list(zip(counts, lens))
        view.used = [0, counts[0], sum(counts)]
        view.held = [[x[:n] for x in h] for h, n in zip(b.held, lens)]
        check(view, q, (out, lse))
    assert att.check() == 0


def test_on_other_streams():
    b = Batch([(1, 3000), (40, 600)], 2, 64, 16)
    q = queries(b, 8, BF)
    want, _ = attend(b, q, 2)
    side = torch.cuda.Stream()
    for current, raw in ((torch.cuda.current_stream(), side.cuda_stream), (side, torch.cuda.default_stream().cuda_stream)):
        with torch.cuda.stream(current):
            att = PagedAttention(8, 2, 64, stream=raw)
            got = att(q, b.cache(), b.sequences(), stream=raw)
            torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_two_workspaces_at_once():
    """Calls on two streams, each with a workspace of its own."""
    b = Batch([(1, 20000), (30, 900)], 2, 64, 16)
    q = queries(b, 8, BF)
    want, _ = attend(b, q, 2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    atts = [PagedAttention(8, 2, 64) for _ in streams]
    cache, seqs = b.cache(), b.sequences()
    outs = [[torch.empty_like(q) for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for st, att, out in zip(streams, atts, outs):
            att(q, cache, seqs, out=out[i], stream=st.cuda_stream)
    torch.cuda.synchronize()
    for out in outs:
        for o in out:
            assert torch.equal(o, want)


def test_places_beyond_32_bits():
    n_pages = (1 << 31) // (16 * 8 * 128) + 40
    cache = PagedCache.empty(n_pages, 16, 8, 128, BF)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    far = Sequences(i32(0, 1, 40), i32(48, 39), i32(n_pages - 1, 0, n_pages - 2, n_pages - 3, n_pages - 4, n_pages - 5).view(2, 3))
    near = Sequences(i32(0, 1, 40), i32(48, 39), i32(1, 2, 3, 4, 5, 6).view(2, 3))
    k, v = (torch.randn(87, 8, 128, device=DEV).to(BF) for _ in range(2))
    q = torch.randn(40, 16, 128, device=DEV).to(BF)
    att, outs = PagedAttention(16, 8, 128), []
    for s in (far, near):
        whole = Sequences(i32(0, 48, 87), i32(48, 39), s.tensors[2])
        cache.write(k, v, whole)
        outs.append(att(q, cache, s))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("cache_type", [BF, E4M3])
def test_a_prompt_in_chunks_then_single_tokens(cache_type):
    """Write, attend, write, attend, as a serving loop does, against attention
    over the whole prompt; and the cache read back."""
    g = torch.Generator(device=DEV).manual_seed(5)
    n, kv_heads, heads, dim, page = 333, 2, 8, 128, 16
    q, k, v = (torch.randn(n, h, dim, generator=g, device=DEV).to(BF) for h in (heads, kv_heads, kv_heads))
    cache = PagedCache.empty(40, page, kv_heads, dim, cache_type)
    table = torch.randperm(40, generator=g, device=DEV).to(torch.int32)[:21].view(1, 21)
    att, at, out = PagedAttention(heads, kv_heads, dim), 0, torch.empty_like(q)
    for rows in (128, 128, 70, 1, 1, 2, 3):
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        seqs = Sequences(i32(0, rows), i32(at + rows), table, max_rows=rows)
        part = slice(at, at + rows)
        cache.write(k[part], v[part], seqs)
        att(q[part], cache, seqs, out=out[part])
        at += rows
    assert at == n
    kc, vc = cache.read(Sequences(torch.tensor([0, n], dtype=torch.int32, device=DEV),
                                  torch.tensor([n], dtype=torch.int32, device=DEV), table), rows=n, out_type=F32)
    torch.cuda.synchronize()
    assert att.check() == 0
    b = Batch([(n, n)], kv_heads, dim, page, cache_type)
    b.held = [[kc.double(), vc.double()]]
    ref, _, d, _ = reference(b, q, dim ** -0.5, True, 0)
    assert ((out.double() - ref).abs() <= d).all()
    if cache_type == BF:
        assert torch.equal(kc, k.float()) and torch.equal(vc, v.float())
    else:  # a code is half of one of 8 steps off, or half the smallest one of the head's scale
        half = k.float().abs() * 2.0 ** -4 + k.float().abs().amax(-1, keepdim=True) / 224 * 2.0 ** -10
        assert ((kc - k.float()).abs() <= half).all()

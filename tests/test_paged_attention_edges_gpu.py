"""Attention over the paged cache at the edges of its contract: device values
outside it, magnitudes far from one, layouts and pages in both kernels."""
import math

import pytest
import torch

from paged import BF, DEV, E4M3, F16, F32, Batch, attend, check, queries, reference
from quantized_routed_expert_gemv_gb300 import moe
from quantized_routed_expert_gemv_gb300.device import PagedAttention, PagedCache, Sequences

pytestmark = pytest.mark.gpu

KINDS = [(BF, BF), (F16, F16), (BF, E4M3), (F16, E4M3)]


# The hint is cut to the rows of the call's tensors: rows of no sequence behind the others
# take calls of few rows to the kernel of many.
def behind(max_rows):
    return 300 if max_rows == 1000 else 0


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("max_rows", [1, 2, 1000])
@pytest.mark.parametrize("starts", [(0, 12, 0, 12), (12, 0, 3, 5), (0, 5, 4, 12), (3, 5, 9, -4), (1 << 30, 0, 12, 12)])
def test_starts_that_fall(max_rows, starts):
    """Nothing is written, and the check says so, once."""
    b = Batch([(4, 300), (4, 20), (4, 700)], 2, 64, 16, max_rows=max_rows)
    q, out, lse = queries(b, 8, BF), torch.full((12, 8, 64), 7.0, dtype=BF, device=DEV), torch.full((12, 8), 7.0, device=DEV)
    good = b.starts.clone()
    att, cache, seqs = PagedAttention(8, 2, 64), b.cache(), b.sequences()
    b.starts.copy_(i32(*starts))
    att(q, cache, seqs, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out == 7.0).all() and (lse == 7.0).all()
    assert att.check() == moe.MOE_ERR_ARG and att.check() == moe.MOE_OK
    b.starts.copy_(good)
    att(q, cache, seqs, out=out, lse=lse)
    torch.cuda.synchronize()
    check(b, q, (out, lse))
    assert att.check() == moe.MOE_OK


@pytest.mark.parametrize("max_rows", [1, 1000])
@pytest.mark.parametrize("n", [129, 600, 65536])
def test_many_starts_that_fall(max_rows, n):
    """Sequences that would have far more tiles together than 32 bits count; and
    one fall among many starts, wherever it is."""
    rows, heads, table = 1024, 8, torch.zeros(n, 256, dtype=torch.int32, device=DEV)
    cache, att = PagedCache.empty(2, 16, heads, 64, BF), PagedAttention(64, heads, 64)
    q = torch.zeros(rows, 64, 64, dtype=BF, device=DEV)
    out = torch.full_like(q, 7.0)
    lens = torch.full((n,), 4096, dtype=torch.int32, device=DEV)
    starts = torch.arange(n + 1, dtype=torch.int32, device=DEV) % 2 * rows
    seqs = Sequences(starts, lens, table, max_rows=max_rows)
    for fall in (None, 1, n // 2, n):
        if fall is not None:
            starts[:fall], starts[fall:] = rows, rows - 1
        att(q, cache, seqs, out=out)
        torch.cuda.synchronize()
        assert (out == 7.0).all() and att.check() == moe.MOE_ERR_ARG


def test_moves_with_starts_that_fall():
    """Rows are taken as some sequence's or none's; nothing else is touched."""
    b = Batch([(4, 8), (4, 8), (4, 8)], 2, 64, 4, BF)
    used = sorted(set(b.table.flatten().tolist()))
    other = [p for p in range(b.n_pages) if p not in used]
    before = b.k[other].clone().view(torch.int16)
    b.starts.copy_(i32(0, 12, 2, 9))
    x = torch.ones(12, 2, 64, dtype=BF, device=DEV)
    k, v = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    cache = b.cache()
    cache.write(x, x, b.sequences())
    cache.read(b.sequences(), k_out=k, v_out=v)
    torch.cuda.synchronize()
    assert torch.equal(b.k[other].view(torch.int16), before)


def test_a_hint_of_single_tokens_for_a_long_prompt():
    """2^31 places of work in tiles of 8 rows: larger ones are taken.  Keys of zeros
    weigh all values alike."""
    n, heads, group, dim = 131072, 8, 8, 16
    cache, att = PagedCache.empty(n // 256, 256, heads, dim, BF), PagedAttention(heads * group, heads, dim)
    cache.tensors[0].zero_(), cache.tensors[1].fill_(0.0)
    cache.tensors[1][:, ::2] = 2.0                               # every second position
    table = torch.arange(n // 256, dtype=torch.int32, device=DEV).view(1, -1)
    q = torch.ones(n, heads * group, dim, dtype=BF, device=DEV)
    out, lse = torch.full_like(q, 7.0), torch.empty(n, heads * group, device=DEV)
    att(q, cache, Sequences(i32(0, n), i32(n), table, max_rows=1), causal=False, out=out, lse=lse)
    torch.cuda.synchronize()
    assert att.check() == 0 and (out == 1.0).all()
    assert (lse - math.log(n)).abs().max().item() <= 2.0 ** -18  # fp32 sums of ones, log2 and a product of 12: 2^-20 each


@pytest.mark.parametrize("code", [0x7F, 0xFF])
@pytest.mark.parametrize("q_type", [BF, F16])
@pytest.mark.parametrize("dim,max_rows", [(64, 1), (64, 1000), (128, 1), (128, 1000), (256, 1000), (80, 1000)])
@pytest.mark.parametrize("scale_up", [0, 12])
def test_codes_that_are_nan_with_finite_scales(code, q_type, dim, max_rows, scale_up):
    """As a cast that does not saturate leaves them.  A key's makes the rows that see it
    NaN, a value's one element of them; the cache read back holds the same."""
    b = Batch([(3, 260)], 2, dim, 16, E4M3, max_rows=max_rows, behind=behind(max_rows))
    if scale_up:  # scales beyond 2^7, which take the second product
        for s in (b.k_scale, b.v_scale):
            s[torch.isfinite(s)] *= 2.0 ** scale_up
        b.held = [[x * 2.0 ** scale_up for x in h] for h in b.held]
    q, scale = queries(b, 4, q_type), dim ** -0.5 * 2.0 ** -scale_up
    clean = attend(b, q, 2, scale=scale)[0][:3]
    check(b, q, attend(b, q, 2, scale=scale), scale=scale)
    element = dim - 3
    for which in "kv":
        for place in (0, 70, 131, 258):
            page, slot = b.table[0, place // 16].item(), place % 16
            at = getattr(b, which).view(torch.uint8)[page, slot, 1]
            kept = at[element].item()
            at[element] = code
            out, lse = (t[:3] for t in attend(b, q, 2, scale=scale))
            ko, vo = b.cache().read(Sequences(i32(0, 260), i32(260), b.table), rows=260, out_type=F32)
            torch.cuda.synchronize()
            assert torch.isnan((ko if which == "k" else vo)[place, 1, element])
            sees = torch.arange(257, 260, device=DEV) >= place
            odd = torch.zeros(3, 4, dim, dtype=torch.bool, device=DEV)
            if which == "k":
                odd[sees, 2:] = True
                assert torch.equal(torch.isnan(lse), odd[..., 0])
            else:
                odd[sees, 2:, element] = True
                assert torch.isfinite(lse).all()
            assert torch.equal(torch.isnan(out), odd)
            d = (out.float() - clean.float()).abs()[~odd]
            # tiles may be taken one position at a time
            assert (d <= 2.0 ** -6 * (2.0 ** scale_up + clean.float().abs()[~odd])).all()
            at[element] = kept


@pytest.mark.parametrize("q_type,cache,power", [
    (BF, BF, 4), (BF, BF, 25), (BF, BF, 33), (BF, BF, 60), (F16, F16, 4), (F16, F16, 25), (F16, F16, 29), (BF, E4M3, 25), (BF, E4M3, 40),
    (F16, E4M3, 25), (F16, E4M3, 29)])
@pytest.mark.parametrize("rows,max_rows,dim", [(1, 1, 64), (3, 2, 128), (3, 1000, 64), (300, 300, 128), (40, 40, 256)])
@pytest.mark.parametrize("scale", [1.0, 0.5])
def test_large_products(q_type, cache, power, rows, max_rows, dim, scale):
    """z of 2^power and a few steps of fp32 below: exact, so the weights are too, but
    for the product with the scale (2^-22 of up to 2^7 steps' logarithm), the
    exponentials (2^-22) and the sum, beside their rounding to 16 bits."""
    length = 700
    b = Batch([(rows, length)], 1, dim, 16, cache, max_rows=max_rows, behind=behind(max_rows))
    step = max(1.0, 2.0 ** (power - 23))                       # z's steps: below 2^power of half of this
    a, k0 = 2.0 ** (power // 2), 2.0 ** (power - power // 2)
    pos = torch.arange(length, device=DEV)
    drop = (1 + (pos * 7) % 5).double()
    k, v = torch.zeros(length, 1, dim, device=DEV, dtype=torch.float64), b.held[0][1].abs() + 0.5
    # z = a k0 - step drop: the second element in units that an e4m3 head of this scale holds
    unit = k0 * 2.0 ** -10
    k[:, 0, 0], k[:, 0, 1] = k0, -drop * unit
    b.held[0] = [b.put(0, "k", pos, k.float() if cache == E4M3 else k), b.put(0, "v", pos, v.float())]
    assert torch.equal(b.held[0][0], k)
    q = torch.zeros(b.rows, 4, dim, device=DEV)
    q[..., 0], q[..., 1] = a, step / unit
    assert torch.equal(q.to(q_type).float(), q)
    out, lse = (t[:rows] for t in attend(b, q.to(q_type), 1, scale=scale, causal=False))
    z = (2.0 ** power - step * drop) * scale
    p = torch.exp(z - z.max())
    want = (p[:, None] * b.held[0][1][:, 0]).sum(0) / p.sum()
    half = 2.0 ** -9 if q_type == BF else 2.0 ** -12
    assert ((out.double() - want).abs() <= want.abs() * (2 * half + 2.0 ** -13)).all()
    assert ((lse.double() - (z.max() + torch.log(p.sum()))).abs() <= 2.0 ** -22 * z.max().abs() + 2.0 ** -13).all()


@pytest.mark.parametrize("q_type,max_rows", [(BF, 1), (F16, 1), (BF, 1000)])
@pytest.mark.parametrize("dim,group", [(64, 1), (128, 4), (80, 8), (256, 2)])
@pytest.mark.parametrize("power", [-60, -20, 20, 40, 100])
@pytest.mark.parametrize("which", ["newest", "newest two", "behind the window", "without weight", "with a small weight", "every other"])
def test_values_of_other_magnitudes(q_type, max_rows, dim, group, power, which):
    """An e4m3 cache, values of some positions 2^power times the others': rows that do
    not see them, or give them (nearly) no weight, are as exact as without them."""
    length, rows, window = 150, 2, 0
    b = Batch([(rows, length), (rows, 40)], 1, dim, 16, E4M3, max_rows=max_rows, behind=behind(max_rows))
    q = queries(b, group, q_type, size=0.5)
    for s, (_, n) in enumerate(b.seqs):
        pos = torch.arange(n, device=DEV)
        k, v = (x.float().clamp(-3, 3) for x in b.held[s])
        k[..., 0] = 0.0
        far = {"newest": pos == n - 1, "newest two": pos >= n - 2, "every other": pos % 2 == 1}.get(which, pos % 16 == 5)
        if which == "behind the window":
            window, far = 21, pos < n - 22
        if which in ("without weight", "with a small weight"):
            # the row's logit is 90 or 30 below: e^-90 < 2^-129, e^-30 about 2^-43
            k[far] = 0.0
            k[far, :, 0] = -90.0 if which == "without weight" else -30.0
            q[..., 0] = 1.0
        v[far] *= 2.0 ** power
        b.held[s] = [b.put(s, "k", pos, k), b.put(s, "v", pos, v)]
    scale = 1.0 if which.startswith("with") and "window" not in which else dim ** -0.5
    # weights of 2^-126 and less of the largest count as nothing: their share of what check() allows
    # for is in its bound only while the values are below 2^70 or so
    if which == "without weight" and power == 100:
        for h in b.held:
            far = torch.arange(len(h[1]), device=DEV) % 16 == 5
            h[1] = torch.where(far[:, None, None], torch.zeros_like(h[1]), h[1])
    out, lse = attend(b, q, 1, scale=scale, window=window)
    out, lse, ref, rlse, d, dl = (t[:2 * rows] for t in (out, lse, *reference(b, q, scale, True, window)))
    # float16 holds magnitudes below 65520; larger ones are infinite
    inside, outside = ref.abs() + d < 65504, ref.abs() - d >= 65520
    if q_type == BF:
        inside, outside = torch.ones_like(inside), torch.zeros_like(outside)
    far = (out.double() - ref).abs() - d
    assert (far[inside] <= 0).all(), f"{far[inside].max().item()} over its bound"
    assert torch.isinf(out[outside]).all() and ((lse.double() - rlse).abs() <= dl).all()


@pytest.mark.parametrize("max_rows", [1, 1000])
@pytest.mark.parametrize("power", [-124, -110, -60, 60, 110])
def test_keys_and_queries_far_apart(max_rows, power):
    """Keys of an e4m3 cache of about 2^power, queries of 2^-power: neither scale may be
    multiplied on z by itself.  One position has a key of zeros."""
    b = Batch([(3, 200), (1, 77)], 2, 128, 16, E4M3, max_rows=max_rows, behind=behind(max_rows))
    for s, (_, n) in enumerate(b.seqs):
        pos = torch.arange(n, device=DEV)
        k = torch.randn(n, 2, 128, device=DEV, generator=torch.Generator(DEV).manual_seed(s)).double().clamp(-3, 3) * 2.0 ** power
        k[7] = 0.0
        b.held[s][0] = b.put(s, "k", pos, k)
    q = (queries(b, 8, F32).double().clamp(-3, 3) * 2.0 ** -power).to(BF)
    check(b, q, attend(b, q, 2))

"""Paged caches, batches and attention in 64 bits, for the tests of the paged
cache and of attention over it: written from the definitions, one sequence at
a time, with the bounds that the kernels' roundings leave."""
import math

import torch

from quantized_routed_expert_gemv_gb300.device import PagedAttention, PagedCache, Sequences

DEV = "cuda:0"
BF, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def quantised(x):
    """(codes' values, scale) of x [..., head_dim] in 64 bits: the smallest power
    of two s >= 2^-126 with max |x| <= 448 s, x / s to nearest even of e4m3."""
    x = x.double()
    amax = x.abs().amax(-1)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -126) / 448.0))
    e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(min=-126.0)
    s = torch.exp2(torch.where(amax > 0, e, torch.zeros_like(e)))
    y = x / s[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
    return torch.round(y / step) * step, s


class Batch:
    """A cache with random contents and the sequences (rows, length) over it.
    Slots of no position hold NaN, and so do the scales."""

    def __init__(self, seqs, kv_heads, dim, page, cache=BF, seed=0, spare=3, first=0, behind=0, layout="head", max_rows=None,
                 wide=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.seqs, self.dim, self.page, self.heads, self.type = seqs, dim, page, kv_heads, cache
        pages = [-(-length // page) for _, length in seqs]
        self.n_pages = sum(pages) + spare
        order = torch.randperm(self.n_pages, generator=g, device=DEV).to(torch.int32)
        self.width = max(pages + [1])
        self.table = torch.full((len(seqs), self.width + wide), -1, dtype=torch.int32, device=DEV)[:, :self.width]
        at = 0
        for s, p in enumerate(pages):
            self.table[s, :p] = order[at:at + p]
            at += p
        starts = [first]
        for rows, _ in seqs:
            starts.append(starts[-1] + rows)
        self.rows, self.used = starts[-1] + behind, starts
        self.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.kv_lens = torch.tensor([length for _, length in seqs], dtype=torch.int32, device=DEV)
        self.max_rows = max([r for r, _ in seqs] + [0]) if max_rows is None else max_rows
        shape = (self.n_pages, kv_heads, page, dim) if layout == "head" else (self.n_pages, page, kv_heads, dim)
        if layout == "wide":   # pages inside a larger tensor
            new = lambda *s, t: torch.zeros(s[0], 2, s[1] + 1, *s[2:], dtype=t, device=DEV)[:, 1, :-1]  # noqa: E731
        else:
            new = lambda *s, t: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
        turn = (lambda t: t.transpose(1, 2)) if layout == "head" else (lambda t: t)
        raw = torch.uint8 if cache == E4M3 else cache
        pages_ = [new(*shape, t=raw) for _ in range(2)]
        for t in pages_:
            t.fill_(0x7F if cache == E4M3 else math.nan)
        self.k, self.v = (turn(t.view(E4M3) if cache == E4M3 else t) for t in pages_)
        self.k_scale = self.v_scale = None
        if cache == E4M3:
            self.k_scale, self.v_scale = (turn(new(*shape[:3], t=F32).fill_(math.nan)) for _ in range(2))
        # what the sequences hold, in 64 bits
        self.held = []
        for s, (_, length) in enumerate(seqs):
            kv = [torch.randn(length, kv_heads, dim, generator=g, device=DEV) for _ in range(2)]
            self.held.append([self.put(s, n, torch.arange(length, device=DEV), x) for n, x in zip("kv", kv)])

    def slots(self, s, pos):
        return self.table[s, pos // self.page].long(), pos % self.page

    def put(self, s, name, pos, x):
        """Stores x at the positions; returns the values that they then stand for."""
        page, slot = self.slots(s, pos)
        t = getattr(self, name)
        if self.type != E4M3:
            t[page, slot] = x.to(self.type)
            return x.to(self.type).double()
        codes, scale = quantised(x)
        t.view(torch.uint8)[page, slot] = codes.float().to(E4M3).view(torch.uint8)
        getattr(self, name + "_scale")[page, slot] = scale.float()
        return codes * scale[..., None]

    def cache(self):
        return PagedCache(self.k, self.v, self.k_scale, self.v_scale)

    def sequences(self):
        return Sequences(self.starts, self.kv_lens, self.table, max_rows=self.max_rows)


def reference(b: Batch, q, scale, causal, window):
    """out, lse in 64 bits and bounds on the kernel's distance from them; rows of
    no sequence NaN.

    The kernel's out: stored half a step of its type (h |out|) off; exponentials
    rounded to that type (h of sum p |v|); z off by the fp32 sum of dim
    products (2^-23 each, as tensor cores may cut instead of rounding), by the
    product with scale * log2(e) and the subtraction of the maximum (2^-22 of
    the largest |z|); exponentials of 2^-22, fp32 sums over the length."""
    half = torch.finfo(q.dtype).eps / 2
    n, heads, dim = q.shape
    group = heads // b.heads
    nan = lambda *s: torch.full(s, math.nan, dtype=torch.float64, device=DEV)  # noqa: E731
    out, lse, d_out, d_lse = nan(n, heads, dim), nan(n, heads), nan(n, heads, dim), nan(n, heads)
    for s, (rows, length) in enumerate(b.seqs):
        if rows == 0:
            continue
        at = slice(b.used[s], b.used[s] + rows)
        k, v = (x.repeat_interleave(group, dim=1) for x in b.held[s])
        pos = torch.arange(length, device=DEV)
        mine = torch.arange(length - rows, length, device=DEV)[:, None]
        sees = (pos <= mine) if causal else torch.ones(rows, length, dtype=torch.bool, device=DEV)
        if window:
            sees = sees & (pos > mine - window)
        z = torch.einsum("thd,lhd->thl", q[at].double(), torch.nan_to_num(k)) * scale
        size = torch.einsum("thd,lhd->thl", q[at].double().abs(), torch.nan_to_num(k).abs()) * scale
        z = z.masked_fill(~sees[:, None, :], -math.inf)
        size = size.masked_fill(~sees[:, None, :], 0.0)
        m = z.amax(-1, keepdim=True) if length else nan(rows, heads, 1)
        m = torch.where(m > -math.inf, m, torch.zeros_like(m))
        p = torch.exp(z - m)
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, torch.zeros_like(p))
        out[at] = torch.einsum("thl,lhd->thd", p, torch.nan_to_num(v))
        lse[at] = (m + torch.log(total))[..., 0]
        worst = size.amax(-1) if length else torch.zeros(rows, heads, dtype=torch.float64, device=DEV)
        dz = worst * ((dim + 4) * 2.0 ** -23 + 2.0 ** -21) + length * 2.0 ** -23 + 2.0 ** -20
        weight = torch.einsum("thl,lhd->thd", p, torch.nan_to_num(v).abs())
        d_out[at] = half * out[at].abs() + weight * (half + 2 * dz[..., None]) * (1 + half) + 2.0 ** -24
        d_lse[at] = dz + 2.0 ** -22 * lse[at].abs()
    return out, lse, d_out, d_lse


def queries(b: Batch, heads, dtype, seed=1, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(b.rows, heads, b.dim, generator=g, device=DEV) * size).to(dtype)


def attend(b: Batch, q, heads_kv, scale=None, causal=True, window=0, stream=None):
    """out and lse with 7 in rows of no sequence."""
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)
    att = PagedAttention(q.shape[1], heads_kv, b.dim)
    att(q, b.cache(), b.sequences(), scale=scale, causal=causal, window=window, out=out, lse=lse, stream=stream)
    torch.cuda.synchronize()
    assert att.check() == 0
    return out, lse


def check(b: Batch, q, got, scale=None, causal=True, window=0):
    out, lse = got
    ref, rlse, d, dl = reference(b, q, b.dim ** -0.5 if scale is None else scale, causal, window)
    none = torch.isnan(rlse)
    assert (out[none] == 7.0).all() and (lse[none] == 7.0).all()
    out, lse, ref, rlse, d, dl = (t[~none] for t in (out, lse, ref, rlse, d, dl))
    empty = torch.isneginf(rlse)
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    assert torch.isfinite(out).all() and torch.isfinite(lse[~empty]).all()
    far = (out.double() - ref).abs() - d
    assert (far <= 0).all(), f"out: {far.max().item()} over its bound, {(far > 0).sum().item()} of {far.numel()}"
    far = ((lse.double() - rlse).abs() - dl)[~empty]
    assert (far <= 0).all(), f"lse: {far.max().item()} over its bound"

"""What is timed of the paged key/value cache and the attention that reads it,
with their plain forms in torch.

A batch holds sequences.  Sequence s has the rows starts[s] to starts[s + 1]
of the call's tensors: its n newest tokens, which stand at the positions
kv_lens[s] - n to kv_lens[s] of the sequence.  Position p is kept in slot
p % page_size of the page page_table[s][p // page_size].

* ``write``: keys and values of new tokens go into the cache, in a 16-bit type
  or as e4m3 codes with one power-of-two scale per token and head.
* ``read``: keys and values of the newest n positions come back as rows.
* ``attn``: attention of the new tokens over the cache, their own keys
  included:
      o = sum_j p_j v_j,  p = softmax_j(scale q . k_j)
  over the positions j that a token sees (causal, or the whole cache; a
  window of the newest ones), with the log of the softmax's sum.

``own = False`` runs the plain forms (elementary torch operations in 32
bits); ``own = True`` the library's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
_PAIRS_MAX = 64 * 128 * 4096 * 14336       # query heads x head size x (token, position) pairs
_READ_MAX = 128 * 1024 * 1024              # values of K of all sequences padded to the longest
_ROWS_MAX = 8192 * 1024                    # values of K in one write or read


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one decoded token of one sequence
        _case("write-1x8x128-e4m3", "write", 1, 1, 300, src="bf16", cache="e4m3"),
        # a ragged batch of chunks with head size 80 and pages of 24 slots, rows inside wider ones
        _case("write-ragged-4x80-f16", "write", 9, 199, 500, kv_heads=4, dim=80, page=24, src="f32", cache="f16",
              ragged=True, pad=16, behind=5),
        # a long prompt, quantised
        _case("write-8192x8x128-e4m3", "write", 2, 4096, 4096, src="bf16", cache="e4m3", page=64),
        # a short sequence is taken out, in 32 bits
        _case("read-61x2x64-f16", "read", 1, 61, 61, kv_heads=2, dim=64, src="f32", cache="f16"),
        # a batch of quantised caches read back for another engine
        _case("read-32-ragged-e4m3", "read", 32, 4096, 4096, src="bf16", cache="e4m3", ragged=True),
        # one decoded token, a short context: latency counts
        _case("decode-1x1000", "attn", 1, 1, 1000),
        # a decode batch over quantised caches, from long to short
        _case("decode-64-ragged-e4m3", "attn", 64, 1, 16384, cache="e4m3", ragged=True),
        # one very long sequence with few heads: the keys have to be split
        _case("decode-1x131072", "attn", 1, 1, 131072, kv_heads=2, group=8, page=128),
        # a decode batch of heads of 256 that see a window of the newest positions
        _case("decode-16-window-f16", "attn", 16, 1, 5000, kv_heads=4, group=2, dim=256, page=32, src="f16", cache="f16",
              window=1024, ragged=True),
        # a chunk of a long prompt
        _case("chunk-128-over-32768", "attn", 1, 128, 32768),
        # chunks, single tokens, an empty sequence and one whose first tokens see nothing, all in one call
        _case("mixed-7-ragged-f16", "attn", 7, 301, 2500, kv_heads=6, group=1, dim=80, page=24, src="f16", cache="f16",
              ragged=True, lse=True, behind=3),
        # the last quarter of a long prompt at once
        _case("prefill-4096-over-16384", "attn", 1, 4096, 16384, page=64, lse=True),
    ]


def _case(name, op, seqs, rows, length, kv_heads=8, group=8, dim=128, page=16, src="bf16", cache="bf16", ragged=False,
          causal=True, window=0, lse=False, pad=0, behind=0):
    """rows, length: of the longest sequence.  pad: values between two rows of
    the inputs; behind: rows after the last sequence's."""
    c = {"op": op, "seqs": seqs, "rows": rows, "len": length, "kv_heads": kv_heads, "dim": dim, "page": page, "src": src,
         "cache": cache, "ragged": ragged, "pad": pad, "behind": behind}
    if op == "attn":
        c.update(group=group, causal=causal, window=window, lse=lse)
    return {"name": name, **c} if name else c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(("write", "read", "attn", "attn", "attn"))
    heads, dim = rng.choice((1, 2, 4, 8, 8, 16)), rng.choice((64, 80, 96, 128, 128, 192, 256))
    page = rng.choice((1, 16, 16, 24, 32, 64, 128, 256))
    half = rng.choice(("bf16", "bf16", "f16"))
    behind, pad = rng.choice((0, 0, 3)), rng.choice((0, 0, 8))
    if op != "attn":
        seqs = _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, min(8192, _ROWS_MAX // (seqs * heads * dim)))
        length = rows if op == "read" else _log_int(rng, rows, min(2 * rows + 100, 16384))
        return _case(None, op, seqs, rows, length, heads, 1, dim, page, rng.choice((half, "f32")),
                     rng.choice((half, "e4m3")), ragged=rng.random() < 0.7, pad=pad, behind=behind)
    seqs = _log_int(rng, 1, 64)
    group = rng.choice((1, 2, 4, 5, 8, 8, 16))
    length = _log_int(rng, 1, min(131072, _READ_MAX // (seqs * heads * dim)))
    rows = 1 if rng.random() < 0.4 else _log_int(
        rng, 1, max(1, min(4096, length + 8, _PAIRS_MAX // (2 * seqs * heads * group * dim * length))))
    window = _log_int(rng, 16, max(16, length)) if rng.random() < 0.3 else 0
    return _case(None, op, seqs, rows, length, heads, group, dim, page, half, rng.choice((half, half, "e4m3")),
                 ragged=rng.random() < 0.6, causal=rng.random() < 0.85, window=window, lse=rng.random() < 0.5, pad=pad,
                 behind=behind)


def _batch(c):
    """Rows and lengths of the case's sequences: the first has the most of
    both; of the others in a ragged batch some have no rows, some one."""
    n, R, L = c["seqs"], c["rows"], c["len"]
    if not c["ragged"]:
        return [R] * n, [L] * n
    rng = random.Random("%d %d %d" % (n, R, L))
    lens = [L] + [max(1, int(L * 64.0 ** -rng.random())) for _ in range(n - 1)]
    if c["op"] == "read":
        return lens, lens
    rows = [R] + [min(rng.choice((1, rng.randint(1, R), R)), lens[s + 1]) for s in range(n - 1)]
    if R > 1 and n > 3:
        rows[2] = 0                                      # a sequence that waits
        rows[3] = min(R, lens[3] + 2)                    # its first tokens see nothing
    return rows, lens


def work(case):
    c = case
    rows, lens = _batch(c)
    if c["op"] != "attn":
        values = 2 * sum(min(r, l) for r, l in zip(rows, lens)) * c["kv_heads"]
        return {"bytes": values * (c["dim"] * (_SIZE[c["src"]] + _SIZE[c["cache"]]) + (4 if c["cache"] == "e4m3" else 0)),
                "flops": 2 * values * c["dim"]}
    pairs = positions = 0
    for r, l in zip(rows, lens):
        first, last = l - r, l - 1
        w = c["window"] if c["window"] else 1 << 40
        if r and c["causal"]:
            # token at position p sees min(p + 1, w) positions, none where p < 0
            lo, hi = max(first, 0), last
            full = max(0, min(hi, w - 1) - lo + 1)       # those that see every position before them
            pairs += full * (2 * lo + full + 1) // 2 + (hi - lo + 1 - full) * min(w, 1 << 30)
            positions += l - max(0, first - w + 1)
        elif r:
            for p in range(first, last + 1):
                pairs += min(l, l - p + w - 1)
            positions += min(l, l - first + w - 1)
    each = c["dim"] * _SIZE[c["cache"]] + (4 if c["cache"] == "e4m3" else 0)
    heads = c["kv_heads"] * c["group"]
    return {"bytes": 2 * positions * c["kv_heads"] * each + sum(rows) * heads * (2 * c["dim"] * _SIZE[c["src"]] + (4 if c["lse"] else 0)),
            "flops": 4 * pairs * heads * c["dim"]}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _rows(count, heads, dim, pad, dtype):
    """[count][heads][dim] view into rows that are `pad` values apart."""
    return torch.empty(count, heads * dim + pad, dtype=dtype, device=DEV)[:, :heads * dim].unflatten(1, (heads, dim))


def _inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *sh: torch.randn(*sh, generator=g, device=DEV)  # noqa: E731
    rows, lens = _batch(c)
    n, H, D, P = c["seqs"], c["kv_heads"], c["dim"], c["page"]
    used, total = sum(rows), sum(rows) + c["behind"]
    width = -(-max(lens) // P)
    pages = [-(-l // P) for l in lens]
    n_pages = sum(pages) + 3
    # every sequence's pages lie anywhere in the cache
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([sum(pages[:s]) for s in range(n)], device=DEV)
    slot = torch.arange(width, device=DEV)
    table = order[(first[:, None] + slot).clamp(max=n_pages - 1)]
    table[slot >= torch.tensor(pages, device=DEV)[:, None]] = -1
    starts = torch.tensor([sum(rows[:s]) for s in range(n + 1)], dtype=torch.int32, device=DEV)
    s = {"case": c, "used": used, "total": total, "max_rows": max(rows), "max_len": max(lens), "starts": starts,
         "kv_lens": torch.tensor(lens, dtype=torch.int32, device=DEV), "table": table}
    # pages hold their slots head by head; a few channels of the keys carry most of them
    chan = torch.where(torch.rand(H, 1, D, generator=g, device=DEV) < 0.03, 4.0, 1.0)
    quant = c["cache"] == "e4m3"
    for name in ("k", "v"):
        page = torch.zeros(n_pages, H, P, D, dtype=torch.uint8 if quant else _TYPES[c["cache"]], device=DEV)
        scale = torch.ones(n_pages, H, P, device=DEV)
        if c["op"] != "write":
            step = max(1, (1 << 26) // (H * P * D))
            for p0 in range(0, n_pages, step):
                p1 = min(n_pages, p0 + step)
                x = rnd(p1 - p0, H, P, D)
                if name == "k":
                    x *= chan
                if quant:
                    _, e = torch.frexp(x.abs().amax(dim=3) / 448.0)
                    scale[p0:p1] = torch.ldexp(torch.ones_like(scale[p0:p1]), e)
                    page[p0:p1] = (x / scale[p0:p1, ..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
                else:
                    page[p0:p1] = x
        s[name] = (page.view(torch.float8_e4m3fn) if quant else page).transpose(1, 2)
        s[name + "_scale"] = scale.transpose(1, 2) if quant else None
    if c["op"] == "write":
        for name in ("k_new", "v_new"):
            s[name] = _rows(total, H, D, c["pad"], _TYPES[c["src"]])
            s[name].copy_(rnd(total, H, D) * torch.exp(0.5 * rnd(total, H, 1)))
            s[name][0, 0] = 0.0                          # a head that gives nothing
    elif c["op"] == "read":
        for name in ("k_out", "v_out"):
            s[name] = _rows(total, H, D, c["pad"], _TYPES[c["src"]]).fill_(7.0)
    else:
        heads = H * c["group"]
        s["q"] = _rows(total, heads, D, c["pad"], _TYPES[c["src"]])
        # from nearly uniform to nearly one-hot
        s["q"].copy_(rnd(total, heads, D) * torch.exp(0.7 * rnd(total, heads, 1) - 0.7))
        s["out"] = torch.full((total, heads, D), 7.0, dtype=_TYPES[c["src"]], device=DEV)
        s["lse"] = torch.full((total, heads), 7.0, device=DEV) if c["lse"] else None
        s["scale"] = D ** -0.5
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from quantized_routed_expert_gemv_gb300 import device
        c = case
        s["cache"] = device.PagedCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["seqs"] = device.Sequences(s["starts"], s["kv_lens"], s["table"], max_rows=s["max_rows"])
        if c["op"] == "attn":
            s["attention"] = device.PagedAttention(c["kv_heads"] * c["group"], c["kv_heads"], c["dim"])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    s = state
    c = s["case"]
    if own:
        if c["op"] == "write":
            s["cache"].write(s["k_new"], s["v_new"], s["seqs"])
            return _held(s)
        if c["op"] == "read":
            s["cache"].read(s["seqs"], k_out=s["k_out"], v_out=s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
        s["attention"](s["q"], s["cache"], s["seqs"], scale=s["scale"], causal=c["causal"], window=c["window"], out=s["out"],
                       lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]} if c["lse"] else {"out": s["out"]}
    return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn}[c["op"]](s)


def _held(s):
    """What the cache holds."""
    names = ("k", "v") + (("k_scale", "v_scale") if s["case"]["cache"] == "e4m3" else ())
    return {n: s[n] for n in names}


def _places(s):
    """Sequence of every row, its place in the sequence's rows, and its position."""
    row = torch.arange(s["used"], device=DEV)
    seq = torch.searchsorted(s["starts"][1:], row, right=True, out_int32=True).long()
    nth = row - s["starts"][seq]
    return seq, nth, s["kv_lens"][seq] - (s["starts"][seq + 1] - s["starts"][seq]) + nth


def _slots(s, seq, pos):
    page = s["table"][seq, pos // s["case"]["page"]].long()
    return page, pos % s["case"]["page"]


def _plain_write(s):
    c = s["case"]
    seq, _, pos = _places(s)
    page, slot = _slots(s, seq, pos.clamp(min=0))
    some = pos >= 0
    page, slot = page[some], slot[some]
    quant = c["cache"] == "e4m3"
    x = torch.stack((s["k_new"][:s["used"]], s["v_new"][:s["used"]])).float()[:, some]
    if quant:
        amax = x.abs().amax(dim=3)
        mant, expo = torch.frexp(amax)             # amax = mant * 2^expo, 0.5 <= mant < 1
        expo = torch.where(mant > 0.875, expo - 8, expo - 9).clamp(min=-126)
        scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), expo), torch.ones_like(amax))
        x = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["k"].view(torch.uint8)[page, slot], s["v"].view(torch.uint8)[page, slot] = x[0], x[1]
        s["k_scale"][page, slot], s["v_scale"][page, slot] = scale[0], scale[1]
    else:
        x = x.to(_TYPES[c["cache"]])
        s["k"][page, slot], s["v"][page, slot] = x[0], x[1]
    return _held(s)


def _values(s, name, page, slot):
    if s["case"]["cache"] != "e4m3":
        return s[name][page, slot].float()
    codes = s[name].view(torch.uint8)[page, slot].view(torch.float8_e4m3fn)
    return codes.float() * s[name + "_scale"][page, slot][..., None]


def _plain_read(s):
    seq, _, pos = _places(s)
    page, slot = _slots(s, seq, pos.clamp(min=0))
    some = (pos >= 0)[:, None, None]
    s["k_out"][:s["used"]] = torch.where(some, _values(s, "k", page, slot), 0.0).to(s["k_out"].dtype)
    s["v_out"][:s["used"]] = torch.where(some, _values(s, "v", page, slot), 0.0).to(s["v_out"].dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _plain_attn(s):
    """All sequences padded to the longest."""
    c = s["case"]
    B, R, L, H, G, D = c["seqs"], s["max_rows"], s["max_len"], c["kv_heads"], c["group"], c["dim"]
    seq, nth, _ = _places(s)
    pos = torch.arange(L, device=DEV)
    page, slot = _slots(s, torch.arange(B, device=DEV)[:, None], pos)
    held = (pos < s["kv_lens"][:, None])[:, :, None, None]
    k = torch.where(held, _values(s, "k", page, slot), 0.0)
    v = torch.where(held, _values(s, "v", page, slot), 0.0)
    count = s["starts"][1:] - s["starts"][:-1]
    i = torch.arange(R, device=DEV)
    at = (s["starts"][:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["q"][at].float().view(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    z = (q @ k.permute(0, 2, 3, 1)).view(B, H, R, G, L) * s["scale"]
    mine = (s["kv_lens"] - count)[:, None, None] + i[:, None]          # [B][R][1]: the tokens' positions
    sees = (pos < s["kv_lens"][:, None, None]).expand(B, R, L)
    if c["causal"]:
        sees = sees & (pos <= mine)
    if c["window"]:
        sees = sees & (pos > mine - c["window"])
    z = z.masked_fill_(~sees[:, None, :, None, :], -math.inf)
    m = z.amax(dim=4, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = z.sub_(m).exp_()
    total = p.sum(dim=4, keepdim=True)
    o = (p.view(B, H, R * G, L) @ v.transpose(1, 2)).view(B, H, R, G, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(B, R, H * G, D)
    s["out"][:s["used"]] = o[seq, nth].to(s["out"].dtype)
    if not c["lse"]:
        return {"out": s["out"]}
    lse = (m + torch.log(total)).permute(0, 2, 1, 3, 4).reshape(B, R, H * G)
    s["lse"][:s["used"]] = lse[seq, nth]
    return {"out": s["out"], "lse": s["lse"]}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    c, s = case, _inputs(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attn": _exact_attn}[c["op"]](c, s)


def _decoded(codes):
    """e4m3 codes as the values they stand for."""
    u = codes.contiguous().view(torch.uint8).to(torch.int32)
    ex, mn = (u >> 3) & 15, (u & 7).double()
    w = torch.where(ex > 0, (8.0 + mn) * torch.exp2(ex.double() - 10.0), mn * 2.0 ** -9)
    return torch.where(u >= 128, -w, w)


def _exact_write(c, s):
    rows, lens = _batch(c)
    quant = c["cache"] == "e4m3"
    out = {}
    for name in ("k", "v"):
        held = torch.zeros(s[name].shape, dtype=torch.float64, device=DEV)
        scales = torch.ones(s[name].shape[:3], dtype=torch.float64, device=DEV)
        row = 0
        for b, (r, l) in enumerate(zip(rows, lens)):
            skip = max(0, r - l)
            x = s[name + "_new"][row + skip:row + r].double()
            pos = torch.arange(l - r + skip, l, device=DEV)
            page, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
            if quant:
                amax = x.abs().max(dim=2).values
                e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -126) / 448.0))
                # the logarithm of a power of two may come out just above it
                e = torch.where(amax <= 448.0 * torch.exp2(e - 1.0), e - 1.0, e).clamp(min=-126.0)
                e = torch.where(amax > 0, e, torch.zeros_like(e))
                x = x * torch.exp2(-e)[..., None]
                # steps of 2^-3 of the value's power of two, 2^-9 below 2^-6
                step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3.0)
                x = torch.round(x / step) * step
                scales[page, slot] = torch.exp2(e)
            held[page, slot] = x
            row += r
        out[name] = held
        if quant:
            out[name + "_scale"] = scales
    return out


def _exact_values(c, s, name, b, pos):
    page, slot = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    if c["cache"] != "e4m3":
        return s[name][page, slot].double()
    return _decoded(s[name].view(torch.uint8)[page, slot]) * s[name + "_scale"][page, slot].double()[..., None]


def _exact_read(c, s):
    rows, lens = _batch(c)
    out = {}
    for name in ("k", "v"):
        parts = [_exact_values(c, s, name, b, torch.arange(l - r, l, device=DEV)) for b, (r, l) in enumerate(zip(rows, lens))]
        parts.append(s[name + "_out"][s["used"]:].double())
        out[name] = torch.cat(parts)
    return out


def _exact_attn(c, s):
    rows, lens = _batch(c)
    H, G, D = c["kv_heads"], c["group"], c["dim"]
    out = s["out"].double()
    lse = torch.full((s["total"], H * G), 7.0, dtype=torch.float64, device=DEV)
    row = 0
    for b, (r, l) in enumerate(zip(rows, lens)):
        pos = torch.arange(l, device=DEV)
        k, v = _exact_values(c, s, "k", b, pos), _exact_values(c, s, "v", b, pos)
        step = max(1, (1 << 27) // (l * G))
        for i0 in range(0, r, step):
            i1 = min(r, i0 + step)
            mine = torch.arange(l - r + i0, l - r + i1, device=DEV)[:, None]
            sees = torch.ones(i1 - i0, l, dtype=torch.bool, device=DEV)
            if c["causal"]:
                sees &= pos <= mine
            if c["window"]:
                sees &= pos > mine - c["window"]
            sees = sees.repeat_interleave(G, dim=0)
            for h in range(H):
                q = s["q"][row + i0:row + i1, h * G:(h + 1) * G].double().reshape(-1, D)
                z = torch.einsum("td,ld->tl", q, k[:, h]) * s["scale"]
                z[~sees] = -math.inf
                total = torch.logsumexp(z, dim=1)
                p = torch.exp(z - torch.where(torch.isinf(total), torch.zeros_like(total), total)[:, None])
                out[row + i0:row + i1, h * G:(h + 1) * G] = torch.einsum("tl,ld->td", p, v[:, h]).view(-1, G, D)
                lse[row + i0:row + i1, h * G:(h + 1) * G] = total.view(-1, G)
        row += r
    return {"out": out, "lse": lse} if c["lse"] else {"out": out}

"""What is timed of the operators around the Mixture-of-Experts layer, with
their plain forms in torch.

Three operators stand between one layer and the next, and between the last
layer and the answer:

* ``norm``: the block boundary.  The block's output y is normalised (RMS),
  gated, added to the scaled residual stream h, and the sum is normalised
  again as the next block's input x:
      r = y * rsqrt(mean(y^2) + eps) * (w_add + w_post)
      h' = residual_scale * h + gate * r
      x  = h' * rsqrt(mean(h'^2) + eps) * (w_add + w_pre)
* ``fp8``: a linear layer in 8-bit floating point (e4m3): weights with one
  float scale per 128 x 128 block, inputs quantised by the call with one
  power-of-two scale per row and block of 128 inputs.
* ``logprobs``: per row of logits the log probabilities and ranks of given
  tokens, the entropy, and the most likely tokens with their log
  probabilities.

``own = False`` runs the plain forms (elementary torch operations in 32
bits); ``own = True`` the library's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_ROWS_MAX_NORM, _H_MAX = 8192, 7168
_W_MAX = 131072 * 7168            # weights of the largest product
_MNK_MAX = 4096 * 7168 * 7168
_LOGITS_MAX = 4096 * 131072


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one decoded token between two large layers: latency counts
        _norm("norm-1x7168", 1, 7168, y="f32", gate="channel"),
        # a decode batch of the mid layer, a gate of its own for each token and channel
        _norm("norm-16x2048", 16, 2048, y="bf16", gate="full"),
        # rows of an odd width inside wider rows, float16 residual stream, a gate per token
        _norm("norm-1021x1999-padded", 1021, 1999, y="f16", h="f16", gate="token", pad=9, w_add=1.0),
        # a long prompt through the large layer
        _norm("norm-8192x7168", 8192, 7168, y="f32", gate="channel"),
        # one decoded token through a square projection of the mid layer
        _fp8("fp8-1x2048x2048", 1, 2048, 2048),
        # a decode batch through the output head of the large layer's width
        _fp8("fp8-head-16x131072x7168", 16, 131072, 7168, out="f32"),
        # a short prompt; nothing divides by 128, float32 inputs and outputs
        _fp8("fp8-77x7000x2003", 77, 7000, 2003, x="f32", out="f32", pad=5),
        # a long prompt through a square projection of the large layer
        _fp8("fp8-4096x7168x7168", 4096, 7168, 7168),
        # one decoded token's logits
        _lp("logprobs-1x131072", 1, 131072, top=20),
        # a batch under grammar masks: most tokens -inf, one row with no token left
        _lp("logprobs-64x50001-masked", 64, 50001, logits="f32", top=8, targets=4, mask="grammar", scale=1.25),
        # a batch whose masks are the type's lowest value, and no alternatives asked
        _lp("logprobs-300x32003-f16", 300, 32003, logits="f16", top=0, mask="lowest", pad=13),
        # every position of a long prompt scored
        _lp("logprobs-4096x131072", 4096, 131072, top=5),
    ]


def _norm(name, rows, hidden, y="bf16", h="bf16", gate="channel", pad=0, w_add=0.0):
    c = {"op": "norm", "rows": rows, "hidden": hidden, "y": y, "h": h, "gate": gate, "pad": pad, "w_add": w_add}
    return {"name": name, **c} if name else c


def _fp8(name, rows, n, k, x="bf16", out="bf16", pad=0):
    c = {"op": "fp8", "rows": rows, "n": n, "k": k, "x": x, "out": out, "pad": pad}
    return {"name": name, **c} if name else c


def _lp(name, rows, vocab, logits="bf16", top=5, targets=1, mask="none", scale=1.0, pad=0):
    c = {"op": "logprobs", "rows": rows, "vocab": vocab, "logits": logits, "top": top, "targets": targets,
         "mask": mask, "scale": scale, "pad": pad}
    return {"name": name, **c} if name else c


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "fp8", "logprobs"))
    kind = lambda: rng.choice(("bf16", "bf16", "f16", "f32"))  # noqa: E731
    if op == "norm":
        hidden = _log_int(rng, 64, 8192)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        rows = _log_int(rng, 1, min(_ROWS_MAX_NORM, _ROWS_MAX_NORM * _H_MAX // hidden))
        return _norm(None, rows, hidden, y=kind(), h=kind() if rows * hidden < 1 << 24 else "bf16",
                     gate=rng.choice(("none", "channel", "token", "full")) if rows * hidden < 1 << 24 else "channel",
                     pad=rng.choice((0, 0, 1, 8)), w_add=rng.choice((0.0, 1.0)))
    if op == "fp8":
        k = _log_int(rng, 64, 7168)
        n = _log_int(rng, 100, min(131072, _W_MAX // k))
        if rng.random() < 0.5:
            k, n = max(64, k // 64 * 64), max(64, n // 64 * 64)
        rows = _log_int(rng, 1, max(1, min(4096, _MNK_MAX // (n * k), (1 << 26) // n)))
        return _fp8(None, rows, n, k, x=kind(), out=kind(), pad=rng.choice((0, 0, 3, 16)))
    vocab = _log_int(rng, 500, 200000)
    kinds = kind()
    rows = _log_int(rng, 1, min(4096, (_LOGITS_MAX // 2 if kinds == "f32" else _LOGITS_MAX * 3 // 4) // vocab))
    mask = rng.choice(("none", "none", "grammar", "lowest"))
    return _lp(None, rows, vocab, logits=kinds, top=rng.choice((0, 1, 5, 20, 32)), targets=rng.choice((1, 1, 2, 8)),
               mask=mask, scale=rng.choice((1.0, 0.7, 1.0 if mask == "lowest" else 1.25)), pad=rng.choice((0, 0, 1, 8)))


def work(case):
    c = case
    if c["op"] == "norm":
        T, H = c["rows"], c["hidden"]
        gate = {"none": 0, "channel": 2 * H, "token": 2 * T, "full": 2 * T * H}[c["gate"]]
        return {"bytes": T * H * (_SIZE[c["y"]] + 2 * _SIZE[c["h"]] + 2) + gate + 4 * H, "flops": 11 * T * H}
    if c["op"] == "fp8":
        M, N, K = c["rows"], c["n"], c["k"]
        return {"bytes": N * K + 4 * _ceil(N) * _ceil(K) + M * K * _SIZE[c["x"]] + M * N * _SIZE[c["out"]],
                "flops": 2 * M * N * K}
    T, V, G, n = c["rows"], c["vocab"], c["targets"], c["top"]
    return {"bytes": T * V * _SIZE[c["logits"]] + T * (12 * G + 8 + 8 * n), "flops": 6 * T * V}


def _ceil(v):
    return -(-v // 128)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _padded(rows, cols, pad, dtype):
    """[rows][cols] view into rows of cols + pad values."""
    return torch.empty(rows, cols + pad, dtype=dtype, device=DEV)[:, :cols]


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"norm": _prepare_norm, "fp8": _prepare_fp8, "logprobs": _prepare_logprobs}[c["op"]](c, g)
    s["case"] = c
    if own:
        {"norm": _own_norm, "fp8": _own_fp8, "logprobs": _own_logprobs}[c["op"]](s)
    return s


def _prepare_norm(c, g):
    T, H, pad = c["rows"], c["hidden"], c["pad"]
    rnd = lambda *sh: torch.randn(*sh, generator=g, device=DEV)  # noqa: E731
    y = _padded(T, H, pad, _TYPES[c["y"]])
    y.copy_(rnd(T, H).mul_(torch.exp(0.5 * rnd(T, 1))))
    # the residual stream: a few channels carry most of it
    h = _padded(T, H, pad, _TYPES[c["h"]])
    chan = torch.where(torch.rand(H, generator=g, device=DEV) < 0.01, 20.0, 1.0)
    h.copy_(rnd(T, H).mul_(chan))
    s = {"y": y, "h": h, "eps": 1e-6, "residual_scale": 0.875}
    for name in ("w_post", "w_pre"):
        s[name] = (1.0 - c["w_add"] + 0.1 * rnd(H)).to(torch.bfloat16)
    shape = {"none": None, "channel": (1, H), "token": (T, 1), "full": (T, H)}[c["gate"]]
    s["gate"] = None if shape is None else torch.rand(*shape, generator=g, device=DEV).add_(0.25).to(torch.bfloat16)
    return s


def _prepare_fp8(c, g):
    M, N, K, pad = c["rows"], c["n"], c["k"], c["pad"]
    x = _padded(M, K, pad, _TYPES[c["x"]])
    x.copy_(torch.randn(M, K, generator=g, device=DEV).mul_(torch.exp(0.5 * torch.randn(M, 1, generator=g, device=DEV))))
    # weights: normal values quantised with one scale per 128 x 128 block
    ld = -(-K // 16) * 16
    codes = torch.zeros(N, ld, dtype=torch.uint8, device=DEV)
    scales = torch.empty(_ceil(N), _ceil(K), dtype=torch.float32, device=DEV)
    step = 16384
    for n0 in range(0, N, step):
        n1 = min(N, n0 + step)
        w = torch.zeros(_ceil(n1 - n0) * 128, _ceil(K) * 128, device=DEV)
        w[:n1 - n0, :K].normal_(0.0, K ** -0.5, generator=g)
        b = w.view(_ceil(n1 - n0), 128, _ceil(K), 128)
        sc = b.abs().amax(dim=(1, 3)) / 448.0
        scales[n0 // 128:_ceil(n1)] = sc
        q = (b / sc[:, None, :, None]).view_as(w).to(torch.float8_e4m3fn)
        codes[n0:n1, :K] = q[:n1 - n0, :K].view(torch.uint8)
    return {"x": x, "codes": codes, "scales": scales}


def _prepare_logprobs(c, g):
    T, V, G = c["rows"], c["vocab"], c["targets"]
    logits = _padded(T, V, c["pad"], _TYPES[c["logits"]])
    sharp = torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV)) * 2.5
    step = max(1, (1 << 26) // V)
    for t0 in range(0, T, step):
        t1 = min(T, t0 + step)
        logits[t0:t1] = torch.randn(t1 - t0, V, generator=g, device=DEV) * sharp[t0:t1]
    targets = torch.randint(0, V, (T, G), generator=g, device=DEV, dtype=torch.int32)
    if c["mask"] != "none":
        low = -math.inf if c["mask"] == "grammar" else torch.finfo(logits.dtype).min
        # the share of tokens that a row's mask leaves: from all to a few
        keep = 10.0 ** (-4.0 * torch.rand(T, 1, generator=g, device=DEV))
        for t0 in range(0, T, step):
            t1 = min(T, t0 + step)
            off = torch.rand(t1 - t0, V, generator=g, device=DEV) > keep[t0:t1]
            logits[t0:t1].masked_fill_(off, low)
        if T > 1:
            logits[T // 2] = low      # one row is left with no token
    # the scored token is often a likely one
    likely = torch.rand(T, 1, generator=g, device=DEV) < 0.7
    targets[:, :1] = torch.where(likely, logits.float().argmax(dim=1, keepdim=True).int() if T * V < 1 << 27
                                 else targets[:, :1], targets[:, :1])
    return {"logits": logits, "targets": targets}


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _call_norm, "fp8": _call_fp8, "logprobs": _call_logprobs}[op](state)
    return {"norm": _plain_norm, "fp8": _plain_fp8, "logprobs": _plain_logprobs}[op](state)


def _plain_norm(s):
    y, h = s["y"].float(), s["h"].float()
    w_add = s["case"]["w_add"]
    r = y * torch.rsqrt(y.square().mean(dim=1, keepdim=True) + s["eps"]) * (w_add + s["w_post"].float())
    if s["gate"] is not None:
        r = r * s["gate"].float()
    hn = s["residual_scale"] * h + r
    x = hn * torch.rsqrt(hn.square().mean(dim=1, keepdim=True) + s["eps"]) * (w_add + s["w_pre"].float())
    return {"h": hn.to(s["h"].dtype), "x": x.to(torch.bfloat16)}


def _plain_fp8(s):
    c = s["case"]
    M, N, K = c["rows"], c["n"], c["k"]
    x = torch.nn.functional.pad(s["x"].float(), (0, _ceil(K) * 128 - K)).view(M, _ceil(K), 128)
    amax = x.abs().amax(dim=2, keepdim=True)
    mant, expo = torch.frexp(amax)             # amax = mant * 2^expo, 0.5 <= mant < 1
    expo = torch.where(mant > 0.875, expo - 8, expo - 9).clamp(min=-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), expo), torch.ones_like(amax))
    xq = ((x / scale).to(torch.float8_e4m3fn).float() * scale).view(M, -1)[:, :K]
    w = s["codes"][:, :K].view(torch.float8_e4m3fn).float()
    rows = torch.arange(N, device=DEV) // 128
    cols = torch.arange(K, device=DEV) // 128
    w = w * s["scales"][rows][:, cols]
    return (xq @ w.t()).to(_TYPES[c["out"]])


def _plain_logprobs(s):
    c = s["case"]
    V, n = c["vocab"], c["top"]
    logits = s["logits"].float()
    x = logits * c["scale"]
    m = x.amax(dim=1, keepdim=True)
    some = m > -math.inf
    e = torch.exp(x - torch.where(some, m, torch.zeros_like(m)))
    total = e.sum(dim=1, keepdim=True)
    lse = m + torch.log(total)
    d = torch.where(e > 0, x - m, torch.zeros_like(x))
    entropy = torch.where(some, torch.log(total) - (e * d).sum(dim=1, keepdim=True) / total, torch.zeros_like(m))
    # differences from the row's maximum first: with logits of the type's lowest value lse alone loses log(total)
    lp = lambda v: torch.where(some & (v > -math.inf), (v - m) - torch.log(total), torch.full_like(v, -math.inf))  # noqa: E731
    t = s["targets"].long()
    xt = logits.gather(1, t)
    # rank: 1 + tokens that come before in (logit descending, id ascending)
    ids = torch.arange(V, device=DEV)
    before = [((logits > xt[:, k:k + 1]) | ((logits == xt[:, k:k + 1]) & (ids < t[:, k:k + 1]))).sum(dim=1)
              for k in range(t.shape[1])]
    out = {"logprob": lp(x.gather(1, t)), "rank": torch.stack(before, dim=1).add(1).int(),
           "entropy": entropy[:, 0], "lse": lse[:, 0]}
    if n:
        # ties go to the lower id: one integer key for value and id
        bits = (logits + 0.0).view(torch.int32).long()
        bits = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF)
        key = bits * (1 << 32) + (V - 1 - ids)
        top = torch.topk(key, min(n, V), dim=1).indices
        xs = x.gather(1, top)
        listed_ = xs > -math.inf
        out["top_ids"] = torch.where(listed_, top, torch.full_like(top, -1)).int()
        out["top_logprobs"] = lp(xs)
    return out


# the library's entry points -------------------------------------------------

def _own_norm(s):
    from quantized_routed_expert_gemv_gb300 import moe
    c = s["case"]
    T, H, pad = c["rows"], c["hidden"], c["pad"]
    s["h_out"] = _padded(T, H, pad, _TYPES[c["h"]])
    s["x_out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    ty = {torch.bfloat16: moe.MOE_BF16, torch.float16: moe.MOE_F16, torch.float32: moe.MOE_F32}
    a = moe.moe_block_norm_args()
    a.rows, a.hidden = T, H
    a.y, a.ld_y, a.y_type = s["y"].data_ptr(), s["y"].stride(0), ty[s["y"].dtype]
    a.h, a.ld_h, a.h_type = s["h"].data_ptr(), s["h"].stride(0), ty[s["h"].dtype]
    if s["gate"] is not None:
        a.gate, a.gate_type = s["gate"].data_ptr(), moe.MOE_BF16
        a.ld_gate_row, a.ld_gate_col = {"channel": (0, 1), "token": (1, 0), "full": (H, 1)}[c["gate"]]
    a.post_norm = a.pre_norm = 1
    a.w_post, a.w_pre, a.w_type = s["w_post"].data_ptr(), s["w_pre"].data_ptr(), moe.MOE_BF16
    a.w_add, a.eps, a.residual_scale = c["w_add"], s["eps"], s["residual_scale"]
    a.h_out, a.ld_h_out = s["h_out"].data_ptr(), s["h_out"].stride(0)
    a.x_out, a.ld_x_out, a.x_type = s["x_out"].data_ptr(), s["x_out"].stride(0), moe.MOE_BF16
    s["args"], s["moe"], s["stream"] = a, moe, torch.cuda.current_stream


def _call_norm(s):
    s["moe"].moe_block_norm(s["args"], s["stream"]().cuda_stream)
    return {"h": s["h_out"], "x": s["x_out"]}


def _own_fp8(s):
    from quantized_routed_expert_gemv_gb300 import device
    c = s["case"]
    s["linear"] = device.Fp8Linear(s["codes"], s["scales"], c["k"], max_rows=c["rows"])
    s["out"] = torch.empty(c["rows"], c["n"], dtype=_TYPES[c["out"]], device=DEV)


def _call_fp8(s):
    return s["linear"](s["x"], s["out"])


def _own_logprobs(s):
    from quantized_routed_expert_gemv_gb300 import moe
    c = s["case"]
    T, V, G, n = c["rows"], c["vocab"], c["targets"], c["top"]
    f32 = lambda *sh: torch.empty(*sh, dtype=torch.float32, device=DEV)  # noqa: E731
    i32 = lambda *sh: torch.empty(*sh, dtype=torch.int32, device=DEV)  # noqa: E731
    o = {"logprob": f32(T, G), "rank": i32(T, G), "entropy": f32(T), "lse": f32(T)}
    if n:
        o["top_ids"], o["top_logprobs"] = i32(T, n), f32(T, n)
    a = moe.moe_token_logprobs_args()
    ty = {torch.bfloat16: moe.MOE_BF16, torch.float16: moe.MOE_F16, torch.float32: moe.MOE_F32}
    a.rows, a.vocab, a.n_targets, a.top_n = T, V, G, n
    a.logits, a.ld_logits, a.logits_type = s["logits"].data_ptr(), s["logits"].stride(0), ty[s["logits"].dtype]
    a.targets, a.scale = s["targets"].data_ptr(), c["scale"]
    a.target_logprobs, a.target_ranks = o["logprob"].data_ptr(), o["rank"].data_ptr()
    a.entropy, a.lse = o["entropy"].data_ptr(), o["lse"].data_ptr()
    if n:
        a.top_ids, a.top_logprobs = o["top_ids"].data_ptr(), o["top_logprobs"].data_ptr()
    s["args"], s["outs"], s["moe"], s["stream"] = a, o, moe, torch.cuda.current_stream


def _call_logprobs(s):
    s["moe"].moe_token_logprobs(s["args"], s["stream"]().cuda_stream)
    return s["outs"]


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    if c["op"] == "norm":
        return _exact_norm(c, _prepare_norm(c, g))
    if c["op"] == "fp8":
        return _exact_fp8(c, _prepare_fp8(c, g))
    return _exact_logprobs(c, _prepare_logprobs(c, g))


def _exact_norm(c, s):
    def rms(v, w):
        return v / torch.sqrt(torch.einsum("th,th->t", v, v)[:, None] / v.shape[1] + s["eps"]) * (w.double() + c["w_add"])
    hs, xs = [], []
    for t0 in range(0, c["rows"], 1024):
        r = rms(s["y"][t0:t0 + 1024].double(), s["w_post"])
        if s["gate"] is not None:
            r *= (s["gate"] if s["gate"].shape[0] == 1 else s["gate"][t0:t0 + 1024]).double()
        hs.append(s["h"][t0:t0 + 1024].double() * s["residual_scale"] + r)
        xs.append(rms(hs[-1], s["w_pre"]))
    return {"h": torch.cat(hs), "x": torch.cat(xs)}


def _exact_fp8(c, s):
    M, N, K = c["rows"], c["n"], c["k"]
    x = s["x"].double()
    out = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    rows = torch.arange(N, device=DEV) // 128
    for kb in range(_ceil(K)):
        k0, k1 = 128 * kb, min(K, 128 * kb + 128)
        b = x[:, k0:k1]
        amax = b.abs().amax(dim=1, keepdim=True)
        p = torch.where(amax > 0, torch.ceil(torch.log2(amax / 448.0)).clamp(min=-126.0), torch.zeros_like(amax))
        v = b * torch.exp2(-p)
        # e4m3: steps of 2^-3 of the value's power of two, 2^-9 below 2^-6
        e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(e - 3.0)
        q = torch.round(v / step) * step * torch.exp2(p)
        u = s["codes"][:, k0:k1].to(torch.int32)
        ex, mn = (u >> 3) & 15, (u & 7).double()
        w = torch.where(ex > 0, (8.0 + mn) * torch.exp2(ex.double() - 10.0), mn * 2.0 ** -9)
        w = torch.where(u >= 128, -w, w) * s["scales"][rows, kb].double()[:, None]
        out += q @ w.t()
    return out


def _exact_logprobs(c, s):
    V, n, T = c["vocab"], c["top"], c["rows"]
    parts = []
    step = max(1, (1 << 26) // V)
    for t0 in range(0, T, step):
        x = s["logits"][t0:t0 + step].double() * float(torch.tensor(c["scale"], dtype=torch.float32))
        most = x.max(dim=1, keepdim=True).values.clamp(min=torch.finfo(torch.float64).min)
        shifted = torch.logsumexp(x - most, dim=1, keepdim=True)
        lse = most + shifted
        l = torch.where(torch.isneginf(x), torch.full_like(x, -math.inf), (x - most) - shifted)
        p = torch.exp(l)
        ent = -torch.where(p > 0, p * l, torch.zeros_like(p)).sum(dim=1)
        part = [l.gather(1, s["targets"][t0:t0 + step].long()), ent, lse[:, 0]]
        if n:
            part.append(torch.topk(l, min(n, V), dim=1).values)
        parts.append(part)
    cols = [torch.cat(p) for p in zip(*parts)]
    out = {"logprob": cols[0], "rank": None, "entropy": cols[1], "lse": cols[2]}
    if n:
        out["top_ids"], out["top_logprobs"] = None, cols[3]
    return out

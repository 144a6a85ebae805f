"""moe_token_logprobs against its definition in 64 bits (numpy).

Tolerance, derived.  With z = scale * l: a thread adds at most
n = 8 ceil(V / 4096) + 8 terms in sequence and the row is joined in at most 16
further additions; a power of two is within 2^-22 and its argument d within
4 * 2^-24 |d|, which moves a term by 4 * 2^-24 |d| ln 2.  Terms are weighted
with p, and sum p |d| ln 2 = sum p |z - scale R| <= spread, where R lies at most
80 ln 2 from the maximum and the mean of |z - max| under p is at most
entropy.  So ln S is within
    e = 2^-24 (n + 16 + 4 + 4 (entropy + 56)).
A log probability adds roundings of its own size (3 * 2^-24 |logprob| and the
product's), lse that of R's, and A / S has the same relative error as S's
terms times their mean distance: entropy is within 3 e (1 + entropy + 56)."""
import numpy as np
import pytest
import torch

from quantized_routed_expert_gemv_gb300 import moe
from quantized_routed_expert_gemv_gb300.device import token_logprobs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
INF = float("inf")


def reference(logits, targets, top_n, scale):
    l = logits.double().cpu().numpy()
    T, V = l.shape
    with np.errstate(over="ignore"):
        z = np.float32(scale).astype(np.float64) * l
        z[np.abs(z) > np.finfo(np.float32).max] = -INF      # overflows to -inf in 32 bits
    out = {k: [] for k in ("lse", "entropy", "logprob", "rank", "top_ids", "top_logprobs")}
    for t in range(T):
        m = z[t].max()
        if m == -INF:
            lp, lse, ent = np.full(V, -INF), -INF, 0.0
        else:
            e = np.exp(z[t] - m)
            s = e.sum()
            lp = (z[t] - m) - np.log(s)
            lse = m + np.log(s)
            p = e / s
            ent = -(p[p > 0] * lp[p > 0]).sum()
        order = np.lexsort((np.arange(V), -l[t]))
        place = np.empty(V, np.int64)
        place[order] = np.arange(V)
        out["lse"].append(lse)
        out["entropy"].append(ent)
        out["logprob"].append([lp[i] if 0 <= i < V else -INF for i in targets[t]])
        out["rank"].append([place[i] + 1 if 0 <= i < V else 0 for i in targets[t]])
        top = [i if z[t, i] > -INF else -1 for i in order[:top_n]] + [-1] * (top_n - min(top_n, V))
        out["top_ids"].append(top)
        out["top_logprobs"].append([lp[i] if i >= 0 else -INF for i in top])
    return {k: np.array(v, np.float64) for k, v in out.items()}


def near(got, want, tol, what):
    got = got.double().cpu().numpy().reshape(want.shape)
    assert np.array_equal(np.isneginf(got), np.isneginf(want)), what
    f = np.isfinite(want)
    tol = np.broadcast_to(tol, want.shape)
    bad = np.abs(got[f] - want[f]) > tol[f]
    assert not bad.any(), (what, got[f][bad][:3], want[f][bad][:3], tol[f][bad][:3])
    assert np.isfinite(got[f]).all(), what


def check(logits, targets=None, top_n=0, scale=1.0, rank=True):
    T, V = logits.shape
    tg = np.zeros((T, 0), np.int64) if targets is None else targets.cpu().numpy().reshape(T, -1)
    ref = reference(logits, tg, top_n, scale)
    out = token_logprobs(logits, targets, top_n=top_n, scale=scale, ranks=rank)
    torch.cuda.synchronize()
    ent = ref["entropy"]
    n = 8 * -(-V // 4096) + 8
    e = 2.0 ** -24 * (n + 20 + 4 * (ent + 56))
    near(out["entropy"], ent, 3 * e * (57 + ent), "entropy")
    fl = np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0)
    near(out["lse"], ref["lse"], e + 2.0 ** -22 * (fl + ent + 1), "lse")
    for name in ("logprob", "top_logprobs"):
        if name in out:
            w = ref[name]
            a = np.where(np.isfinite(w), np.abs(w), 0)
            near(out[name], w, e[:, None] + 2.0 ** -22 * (a + fl[:, None] + 1), name)
    if "rank" in out:
        assert np.array_equal(out["rank"].cpu().numpy().reshape(T, -1), ref["rank"])
    if top_n:
        assert np.array_equal(out["top_ids"].cpu().numpy(), ref["top_ids"])
    return out


def rnd(T, V, dtype=BF, seed=0, scale=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(T, V, generator=g, device=DEV) * scale).to(dtype)


def some_targets(T, V, G, seed=9):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(0, V, (T, G), generator=g, device=DEV, dtype=torch.int32)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 31, 500, 4095, 4096, 4097, 8192, 32003, 65536, 131072])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T", [1, 5])
def test_vocabularies_and_types(T, V, dtype):
    check(rnd(T, V, dtype), some_targets(T, V, 1), top_n=min(20, 32))


@pytest.mark.parametrize("T", [2, 40, 80, 152, 200])
def test_rows_over_the_split_rule(T):
    check(rnd(T, 8500, seed=T), some_targets(T, 8500, 2), top_n=3)


@pytest.mark.parametrize("T,V,dtype", [(2, 131072, BF), (20, 131073, BF), (38, 70001, BF), (77, 70001, HF), (152, 66000, BF),
                                       (153, 66000, BF), (20, 40003, F32), (3, 200000, F32)])
def test_long_rows_in_parts(T, V, dtype):
    """Rows that 2, 4 or 8 blocks share, and the first count of rows that they do not."""
    check(rnd(T, V, dtype, seed=T), some_targets(T, V, 3), top_n=9)


@pytest.mark.parametrize("dtype,V", [(BF, 140001), (F32, 66001)])
def test_long_rows_in_parts_with_masks_and_ties(dtype, V):
    l = rnd(6, V, dtype)
    l[0] = -INF
    l[1] = -INF
    l[1, V - 3] = 1.0                   # one token, in the last part
    l[2] = torch.finfo(dtype).min
    l[3] = 0.5                          # all equal
    l[4, V // 2:] = -INF                # whole parts without a token
    l[5].copy_(torch.arange(V, device=DEV) % 7)
    check(l, some_targets(6, V, 2), top_n=32)


@pytest.mark.parametrize("G", [1, 2, 7, 8])
@pytest.mark.parametrize("top_n", [0, 1, 32])
def test_targets_and_top(G, top_n):
    check(rnd(6, 20001, F32), some_targets(6, 20001, G), top_n=top_n, scale=0.6)


@pytest.mark.parametrize("pad", [1, 3, 8, 13])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides_and_bases(pad, dtype):
    T, V = 7, 5003
    wide = rnd(T, V + pad, dtype)
    wide[:, V:] = 1000.0            # what lies between the rows takes no part
    check(wide[:, :V], some_targets(T, V, 3), top_n=5)
    buf = rnd(1, T * V + 1, dtype)[0]
    check(buf[1:].view(T, V), some_targets(T, V, 3), top_n=5)


@pytest.mark.parametrize("V", [33, 5000, 40000])
def test_ties_go_to_the_lower_id(V):
    g = torch.Generator(device=DEV).manual_seed(3)
    l = torch.randint(-2, 3, (9, V), generator=g, device=DEV).to(BF)
    l[0] = 0.0
    l[1] = -0.0
    l[2, ::2] = -0.0
    l[3] = torch.arange(V, device=DEV).to(BF)
    l[4] = -torch.arange(V, device=DEV).to(BF)
    check(l, some_targets(9, V, 4), top_n=32)


def test_top_tokens_of_one_group():
    """All of the best tokens among those one thread visits: more candidates
    than the buffer holds."""
    V = 300000
    l = rnd(1, V, F32, scale=0.5).repeat(160, 1)
    ids = torch.arange(V, device=DEV)
    l[0, (ids // 8) % 512 == 17] += 50.0
    for q in range(32):
        l[1, (ids // 8) % 512 == 11 * q] += 50.0 + 0.01 * q
    check(l[:2].contiguous(), some_targets(2, V, 1), top_n=32)
    check(l, some_targets(160, V, 1), top_n=32)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("V", [300, 70001])
def test_masks(dtype, V):
    low = torch.finfo(dtype).min
    for fill, scale in ((-INF, 1.3), (low, 1.0)):
        l = rnd(8, V, dtype)
        keep = torch.rand(8, V, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
        for t, share in enumerate((1.0, 0.5, 0.01, 0.001)):
            l[t, keep[t] > share] = fill
        l[4] = fill                     # nothing left
        l[5] = fill
        l[5, V - 1] = 2.0               # one token left
        l[6, :V - 2] = fill
        l[7, 0] = fill
        tg = some_targets(8, V, 3)
        tg[5, 0], tg[5, 1] = V - 1, 0
        check(l, tg, top_n=12, scale=scale)


def test_lowest_values_that_overflow_under_the_scale():
    l = rnd(3, 9000, F32)
    l[0, 10:] = torch.finfo(F32).min
    l[1] = torch.finfo(F32).min
    check(l, some_targets(3, 9000, 2), top_n=12, scale=2.0)


def test_targets_outside_the_vocabulary():
    l = rnd(4, 1000)
    tg = torch.tensor([[-1, 5], [1000, 999], [2 ** 31 - 1, 0], [-2 ** 31, 3]], dtype=torch.int32, device=DEV)
    check(l, tg, top_n=1)


def test_wide_range_of_logits():
    """Logits that rise along the row by thousands: the reference moves."""
    V = 20000
    l = torch.linspace(-3000, 3000, V, device=DEV).repeat(3, 1)
    l[1] = l[1].flip(0)
    l[2] = l[2][torch.randperm(V, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2))]
    check(l, some_targets(3, V, 2), top_n=8)


def test_nan_and_inf():
    l = rnd(4, 6000)
    l[1, 4321] = float("nan")
    l[2, 77] = INF
    l[3, :] = float("nan")
    tg = some_targets(4, 6000, 1)
    out = {k: v.cpu() for k, v in token_logprobs(l, tg, top_n=3).items()}
    for t in (1, 2, 3):
        assert out["lse"][t].isnan() and out["entropy"][t].isnan() and out["logprob"][t].isnan().all()
    assert torch.isfinite(out["lse"][0])
    assert 4321 not in out["top_ids"][1] and out["top_logprobs"][1].isnan().all()
    assert out["top_ids"][2, 0] == 77
    assert (out["top_ids"][3] == -1).all() and (out["top_logprobs"][3] == -INF).all()


def test_optional_outputs_streams_and_repeat():
    l, tg = rnd(20, 40000), some_targets(20, 40000, 2)
    full = check(l, tg, top_n=10)
    some = check(l, tg, rank=False)
    assert torch.equal(full["logprob"], some["logprob"]) and torch.equal(full["lse"], some["lse"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    again = token_logprobs(l, tg, top_n=10, stream=st.cuda_stream)
    st.synchronize()
    for k in full:
        assert torch.equal(full[k], again[k]), k
    none = token_logprobs(l[:0])
    assert none["lse"].shape == (0,)


def test_a_row_past_two_to_the_31_elements():
    """Rows whose offset does not fit 32 bits."""
    V, ld = 4099, (1 << 30) + 8
    buf = torch.empty(3 * ld, dtype=BF, device=DEV)
    l = buf.as_strided((3, V), (ld, 1))
    l.copy_(rnd(3, V))
    check(l, some_targets(3, V, 1), top_n=4)


def test_refuses():
    l = rnd(2, 100)
    for kw in (dict(top_n=33), dict(scale=0.0), dict(scale=float("nan")), dict(scale=INF)):
        with pytest.raises(moe.MoEError) as e:
            token_logprobs(l, **kw)
        assert e.value.code == moe.MOE_ERR_ARG

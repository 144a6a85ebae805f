"""moe_token_logprobs on more rows than four an SM, where blocks of 128 threads
or copies through shared memory read a row, and in small parts of rows, against
its definition in 64 bits.

Few different rows are repeated, so that the definition is worked out once a
row.  The tolerance is the one derived for fewer rows, with the sequence of a
thread of a block of 128 in it: n = 8 ceil(V / 2048) + 8 terms."""
import numpy as np
import pytest
import torch

from quantized_routed_expert_gemv_gb300.device import token_logprobs
from test_token_logprobs_gpu import BF, DEV, F32, HF, INF, near, reference, rnd, some_targets

pytestmark = pytest.mark.gpu


def many(distinct):
    """Repeats of `distinct` rows that make a few more rows than four an SM."""
    return -(-(4 * torch.cuda.get_device_properties(0).multi_processor_count + 3) // distinct)


def check(few, targets=None, top_n=0, scale=1.0, pad=0):
    D, V = few.shape
    R = many(D)
    logits = torch.full((D * R, V + pad), 1000.0, dtype=few.dtype, device=DEV)[:, :V]
    logits.copy_(few.repeat(R, 1))
    tg = np.zeros((D, 0), np.int64) if targets is None else targets.cpu().numpy()
    ref = {k: np.concatenate([v] * R) for k, v in reference(few, tg, top_n, scale).items()}
    out = token_logprobs(logits, None if targets is None else targets.repeat(R, 1), top_n=top_n, scale=scale)
    torch.cuda.synchronize()
    ent = ref["entropy"]
    e = 2.0 ** -24 * (8 * -(-V // 2048) + 8 + 20 + 4 * (ent + 56))
    near(out["entropy"], ent, 3 * e * (57 + ent), "entropy")
    fl = np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0)
    near(out["lse"], ref["lse"], e + 2.0 ** -22 * (fl + ent + 1), "lse")
    for name in ("logprob", "top_logprobs"):
        if name in out:
            w = ref[name]
            a = np.where(np.isfinite(w), np.abs(w), 0)
            near(out[name], w, e[:, None] + 2.0 ** -22 * (a + fl[:, None] + 1), name)
    if targets is not None:
        assert np.array_equal(out["rank"].cpu().numpy(), ref["rank"])
    if top_n:
        assert np.array_equal(out["top_ids"].cpu().numpy(), ref["top_ids"])


@pytest.mark.parametrize("V", [1, 7, 8, 129, 1000, 4099, 8193, 12287, 12288, 13003, 32003, 57344, 57345, 70001])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_vocabularies_and_types(V, dtype):
    check(rnd(6, V, dtype), some_targets(6, V, 1), top_n=20)


@pytest.mark.parametrize("G", [0, 2, 4, 7, 8])
@pytest.mark.parametrize("V", [5003, 20001, 60001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_targets(G, V, dtype):
    check(rnd(5, V, dtype), some_targets(5, V, G) if G else None, top_n=3, scale=0.6)


@pytest.mark.parametrize("pad", [1, 3, 8, 13])
@pytest.mark.parametrize("V", [2003, 14003, 60003])
def test_strides(pad, V):
    check(rnd(7, V), some_targets(7, V, 8), top_n=5, pad=pad)


@pytest.mark.parametrize("V", [33, 5000, 20000, 60000])
def test_ties_go_to_the_lower_id(V):
    g = torch.Generator(device=DEV).manual_seed(3)
    l = torch.randint(-2, 3, (6, V), generator=g, device=DEV).to(BF)
    l[0] = 0.0
    l[1] = -0.0
    l[2, ::2] = -0.0
    l[3] = torch.arange(V, device=DEV).to(BF)
    l[4] = -torch.arange(V, device=DEV).to(BF)
    check(l, some_targets(6, V, 4), top_n=32)


@pytest.mark.parametrize("V,threads", [(57000, 128), (130000, 256)])
def test_top_tokens_of_few_groups(V, threads):
    """More candidates than the buffer holds: the best tokens are those that
    four threads visit."""
    l = rnd(2, V, BF, scale=0.5)
    ids = torch.arange(V, device=DEV)
    for q in range(4):
        l[0, (ids // 8) % threads == 11 * q + 5] += 50.0
    l[1, (ids // 8) % threads == 17] += 50.0
    check(l, some_targets(2, V, 1), top_n=32)


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("V", [300, 13000, 58000])
def test_masks(dtype, V):
    for fill, scale in ((-INF, 1.3), (torch.finfo(dtype).min, 1.0)):
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


@pytest.mark.parametrize("V", [6000, 14000, 60000])
def test_nan_and_inf(V):
    l = rnd(4, V)
    l[1, V - 9] = float("nan")
    l[2, 77] = INF
    l[3, :] = float("nan")
    R = many(4)
    out = {k: v.cpu() for k, v in token_logprobs(l.repeat(R, 1), some_targets(4, V, 1).repeat(R, 1), top_n=3).items()}
    for t in range(4 * R):
        if t % 4 == 0:
            assert torch.isfinite(out["lse"][t])
            continue
        assert out["lse"][t].isnan() and out["entropy"][t].isnan() and out["logprob"][t].isnan().all()
        if t % 4 == 1:
            assert V - 9 not in out["top_ids"][t]
        if t % 4 == 2:
            assert out["top_ids"][t, 0] == 77
        if t % 4 == 3:
            assert (out["top_ids"][t] == -1).all()


def test_repeats_give_the_same_bits():
    l, tg = rnd(3, 20001).repeat(many(3), 1), some_targets(3, 20001, 2).repeat(many(3), 1)
    a, b = (token_logprobs(l, tg, top_n=10) for _ in range(2))
    for k in a:
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("T,V,dtype", [(1, 49152, BF), (37, 50001, HF), (38, 50001, BF), (76, 50001, BF), (77, 50001, BF),
                                       (2, 24577, F32), (75, 33000, F32), (76, 70003, BF), (3, 131072, BF)])
def test_parts_of_16_kb(T, V, dtype):
    """Rows in 2, 4 or 8 parts, around the counts of rows where that changes."""
    l, tg = rnd(T, V, dtype, seed=V), some_targets(T, V, 2)
    l[0, V // 3:] = -INF
    ref = reference(l, tg.cpu().numpy(), 32, 1.0)
    out = token_logprobs(l, tg, top_n=32)
    ent = ref["entropy"]
    e = 2.0 ** -24 * (8 * -(-V // 4096) + 8 + 20 + 4 * (ent + 56))
    near(out["entropy"], ent, 3 * e * (57 + ent), "entropy")
    near(out["lse"], ref["lse"], e + 2.0 ** -22 * (np.abs(ref["lse"]) + ent + 1), "lse")
    assert np.array_equal(out["rank"].cpu().numpy(), ref["rank"])
    assert np.array_equal(out["top_ids"].cpu().numpy(), ref["top_ids"])


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("T,V", [(3, 5001), (2, 131072), (700, 5001), (700, 20001)])
def test_a_nan_target_has_rank_1(T, V, dtype):
    l = rnd(T, V, dtype)
    tg = some_targets(T, V, 2)
    tg[:, 1] = (tg[:, 0] + 1) % V
    rows = torch.arange(T, device=DEV)
    l[rows, tg[:, 0].long()] = float("nan")
    out = token_logprobs(l, tg, top_n=2)
    other = l[rows, tg[:, 1].long()].float()[:, None]
    above = (l.float() > other).sum(1)
    assert (out["rank"][:, 0] == 1).all()
    assert (out["rank"][:, 1] > above).all()            # NaNs come before no target
    assert out["logprob"].isnan().all() and not (out["top_ids"] == tg[:, :1]).any()


@pytest.mark.parametrize("bits", [0x7F800001, 0xFF800001, 0x7FFFFFFF, 0xFFFFFFFF])
def test_any_nan_target_has_rank_1(bits):
    """NaNs next to the infinities too: no step from their bits may reach them."""
    l = rnd(4, 5001, F32)
    l[1] = INF
    l[2] = -INF
    tg = some_targets(4, 5001, 1)
    l.view(torch.int32)[torch.arange(4, device=DEV), tg[:, 0].long()] = bits - (1 << 32) if bits >> 31 else bits
    assert l.isnan().sum() == 4
    assert (token_logprobs(l, tg)["rank"] == 1).all()

"""Refusals of the paged cache and of attention over it (include/moe_cache.h) and
of their tensor wrappers: arguments are checked on the host before any launch,
so these need no GPU."""
import contextlib
import ctypes

import pytest
import torch

from quantized_routed_expert_gemv_gb300 import build, device, moe


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


P = 1 << 20      # an aligned address; validation never reads through it
ARG, ALIGN, OK, UNSUPPORTED = moe.MOE_ERR_ARG, moe.MOE_ERR_ALIGN, moe.MOE_OK, moe.MOE_ERR_UNSUPPORTED


def cache_of(**kw):
    c = moe.moe_kv_cache()
    c.k = c.v = c.k_scale = c.v_scale = P
    c.page_stride, c.slot_stride, c.head_stride = 16 * 2 * 64, 64, 16 * 64
    c.scale_page_stride, c.scale_slot_stride, c.scale_head_stride = 32, 1, 16
    c.type, c.n_pages, c.page_size, c.kv_heads, c.head_dim = moe.MOE_BF16, 4, 16, 2, 64
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def seqs_of(**kw):
    s = moe.moe_sequences()
    s.starts = s.kv_lens = s.page_table = P
    s.ld_table, s.n_seqs, s.rows, s.max_rows, s.table_width = 4, 2, 3, 2, 4
    for k, v in kw.items():
        setattr(s, k, v)
    return s


SHARED = [
    (dict(type=2), {}, ARG), (dict(type=4), {}, ARG), (dict(type=-1), {}, ARG), (dict(head_dim=0), {}, ARG),
    (dict(head_dim=72), {}, ARG), (dict(head_dim=272), {}, ARG), (dict(kv_heads=0), {}, ARG), (dict(kv_heads=1025), {}, ARG),
    (dict(page_size=0), {}, ARG), (dict(page_size=(1 << 20) + 1), {}, ARG), (dict(n_pages=-1), {}, ARG),
    (dict(page_stride=-8), {}, ARG), (dict(slot_stride=68), {}, ARG), (dict(head_stride=4), {}, ARG),
    (dict(type=3, page_stride=2056), {}, ARG), (dict(k=None), {}, ARG), (dict(v=None), {}, ARG), (dict(k=P + 8), {}, ALIGN),
    (dict(v=P + 2), {}, ALIGN), (dict(type=3, k_scale=None), {}, ARG), (dict(type=3, v_scale=None), {}, ARG),
    (dict(type=3, k_scale=P + 2), {}, ALIGN), (dict(type=3, scale_slot_stride=-1), {}, ARG),
    ({}, dict(n_seqs=-1), ARG), ({}, dict(n_seqs=65537), ARG), ({}, dict(rows=-1), ARG), ({}, dict(rows=(1 << 24) + 1), ARG),
    ({}, dict(max_rows=-1), ARG), ({}, dict(table_width=5), ARG), ({}, dict(table_width=-1), ARG), ({}, dict(starts=None), ARG),
    ({}, dict(kv_lens=None), ARG), ({}, dict(page_table=None), ARG), ({}, dict(starts=P + 2), ALIGN),
    ({}, dict(kv_lens=P + 1), ALIGN), ({}, dict(page_table=P + 3), ALIGN), ({}, dict(rows=0), OK), ({}, dict(n_seqs=0), OK)]


@pytest.mark.parametrize("call", ["moe_cache_write", "moe_cache_read"])
@pytest.mark.parametrize("c,s,rc", SHARED)
def test_moves_refuse(L, call, c, s, rc):
    fn = getattr(L, call)
    args = (ctypes.byref(cache_of(**c)), ctypes.byref(seqs_of(**s)), P, 128, P, 128, moe.MOE_F32, None)
    assert fn(*args) == rc
    if rc:
        assert call in moe.last_error()


@pytest.mark.parametrize("call", ["moe_cache_write", "moe_cache_read"])
@pytest.mark.parametrize("k,ld_k,v,ld_v,t,rc", [
    (None, 128, P, 128, 0, ARG), (P, 128, None, 128, 0, ARG), (P, 127, P, 128, 0, ARG), (P, 128, P, 0, 0, ARG),
    (P, 128, P, 128, 3, ARG), (P, 128, P, 128, -1, ARG), (P + 1, 128, P, 128, 0, ALIGN), (P, 128, P + 2, 128, 2, ALIGN)])
def test_moves_refuse_rows(L, call, k, ld_k, v, ld_v, t, rc):
    fn = getattr(L, call)
    assert fn(ctypes.byref(cache_of()), ctypes.byref(seqs_of()), k, ld_k, v, ld_v, t, None) == rc
    assert call in moe.last_error()
    assert fn(None, ctypes.byref(seqs_of()), P, 128, P, 128, 0, None) == ARG
    assert fn(ctypes.byref(cache_of()), None, P, 128, P, 128, 0, None) == ARG


def test_too_many_threads_are_refused(L):
    c = cache_of(kv_heads=1024, head_dim=256, head_stride=16 * 256, slot_stride=256)
    assert L.moe_cache_write(ctypes.byref(c), ctypes.byref(seqs_of(rows=1 << 24)), P, 1 << 18, P, 1 << 18, 0, None) == ARG


def attn_args(**kw):
    a = moe.moe_attention_args()
    a.q = a.out = a.lse = P
    a.ld_q = a.ld_out = 4 * 64
    a.q_type, a.q_heads, a.causal, a.window, a.scale = moe.MOE_BF16, 4, 1, 0, 0.125
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("c,s,rc", SHARED)
def test_attention_refuses_caches(L, c, s, rc):
    assert L.moe_attention(ctypes.byref(attn_args()), ctypes.byref(cache_of(**c)), ctypes.byref(seqs_of(**s)), P, 1 << 30,
                           None) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(q_type=2), ARG), (dict(q_type=3), ARG), (dict(q_type=1), UNSUPPORTED), (dict(q_heads=3), ARG), (dict(q_heads=0), ARG),
    (dict(q_heads=-2), ARG), (dict(q_heads=258, ld_q=1 << 20, ld_out=1 << 20), ARG), (dict(q_heads=4098), ARG),
    (dict(causal=2), ARG), (dict(causal=-1), ARG), (dict(window=-1), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(q=None), ARG), (dict(out=None), ARG),
    (dict(ld_q=255), ARG), (dict(ld_q=260), ARG), (dict(ld_out=248), ARG), (dict(ld_out=257), ARG), (dict(q=P + 2), ALIGN),
    (dict(out=P + 8), ALIGN), (dict(lse=P + 2), ALIGN)])
def test_attention_refuses(L, kw, rc):
    call = lambda a, ws=P: L.moe_attention(ctypes.byref(a), ctypes.byref(cache_of()), ctypes.byref(seqs_of()), ws, 1 << 30, None)  # noqa: E731
    assert call(attn_args(**kw)) == rc
    assert "moe_attention" in moe.last_error()
    assert call(attn_args(), None) == ARG and call(attn_args(), P + 128) == ALIGN
    assert L.moe_attention(None, ctypes.byref(cache_of()), ctypes.byref(seqs_of()), P, 1 << 30, None) == ARG
    many = seqs_of(rows=1 << 24)
    wide = attn_args(q_heads=256, ld_q=256 * 64, ld_out=256 * 64)
    assert L.moe_attention(ctypes.byref(wide), ctypes.byref(cache_of()), ctypes.byref(many), P, 1 << 30, None) == ARG


def test_more_work_than_counts_is_refused(L):
    c = cache_of(page_size=1 << 20)
    s = seqs_of(n_seqs=65536, rows=65536, table_width=1024, ld_table=1024)
    assert L.moe_attention(ctypes.byref(attn_args()), ctypes.byref(c), ctypes.byref(s), P, 1 << 30, None) == UNSUPPORTED


# rows, sequences, table width (of pages of 16), heads, head size, max_rows: a workspace of 0 bytes is
# refused after the count of the work, so nothing is launched
@pytest.mark.parametrize("rows,n,width,heads,dim,max_rows,fits", [
    # one prompt of 262144: 2^31 tiles of 16 rows and 64 positions, 1/32 of that in tiles of 256 and 128
    (262144, 1, 16384, (64, 8), 128, 262144, True),
    # the hint of single tokens is wrong: tiles of 8 rows would be too many, larger ones are not
    (131072, 1, 8192, (64, 8), 128, 1, True), (1 << 20, 1, 8192, (64, 8), 128, 1, True),
    # both sides of the limit: (2^15 * 4 / 128 + n) * 1 * (2^24 / 64 + 4) <= 2^31 - 1
    (1 << 15, 7167, 1 << 20, (4, 1), 256, 1000, True), (1 << 15, 7168, 1 << 20, (4, 1), 256, 1000, False),
    (1 << 15, 7168, 1 << 20, (4, 1), 256, 1, False),
    # and of the larger tiles: (2^20 * 4 / 256 + n) * 1 * (2^24 / 128 + 4)
    (1 << 20, 0, 1 << 20, (4, 1), 64, 9, True), (1 << 15, 15871, 1 << 20, (4, 1), 64, 1, True),
    (1 << 15, 15872, 1 << 20, (4, 1), 64, 1, False)])
def test_the_work_that_counts(L, rows, n, width, heads, dim, max_rows, fits):
    if fits and n:
        assert (rows * heads[0] // heads[1] // (256 if dim <= 128 else 128) + n) * heads[1] * (width * 16 // (128 if dim <= 128 else 64) + 4) < 2 ** 31
    c = cache_of(kv_heads=heads[1], head_dim=dim, head_stride=16 * dim, slot_stride=dim, page_stride=16 * dim * heads[1])
    a = attn_args(q_heads=heads[0], ld_q=heads[0] * dim, ld_out=heads[0] * dim)
    s = seqs_of(n_seqs=n, rows=rows, table_width=width, ld_table=width, max_rows=max_rows)
    rc = L.moe_attention(ctypes.byref(a), ctypes.byref(c), ctypes.byref(s), P, 0, None)
    assert (rc != UNSUPPORTED) == fits and (rc != OK or n == 0)


def test_calls_on_another_stream(calls, monkeypatch):
    """What a call on another stream uses is recorded on it, and what it allocates is its own."""
    used, asked = [], []

    class Other:
        def __init__(self, raw):
            self.raw = raw

    monkeypatch.setattr(device, "_other", lambda dev, st: None if st in (None, 0) else Other(st))
    monkeypatch.setattr(device, "_empty", lambda dev, other, dtype, *shape: asked.append(other) or torch.empty(*shape, dtype=dtype))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, st: used.append(st.raw))
    monkeypatch.setattr(torch.cuda, "stream", lambda st: contextlib.nullcontext())
    c, s = a_cache(torch.float8_e4m3fn), some_seqs()
    att = device.PagedAttention(4, 2, 64, device=_Cpu(), stream=5)
    assert asked[-1].raw == 5
    q, k = Z(3, 4, 64, dtype=BF), Z(3, 2, 64, dtype=BF)
    for call, own in ((lambda st: c.write(k, k, s, stream=st), 7), (lambda st: c.read(s, rows=3, stream=st), 7),
                      (lambda st: att(q, c, s, stream=st), 8)):
        del used[:], asked[:]
        call(9)
        assert used == [9] * own and all(o.raw == 9 for o in asked)
        assert calls[-1][1][-1] == 9
        del used[:], asked[:]
        call(None)
        assert used == [] and all(o is None for o in asked)


def test_workspaces_refuse(L):
    for heads in ((0, 1, 64), (4, 0, 64), (3, 2, 64), (4, 2, 72), (4, 2, 0), (258, 2, 64), (4, 2, 512)):
        assert L.moe_attention_workspace_bytes(*heads) == 0
    assert L.moe_attention_workspace_init(None, 1 << 20, None) == ARG
    assert L.moe_attention_workspace_init(P, 255, None) == ARG
    assert L.moe_attention_workspace_init(P + 16, 1 << 20, None) == ALIGN
    assert L.moe_attention_check(None, None) == ARG


# ---- the tensor wrappers, with the library replaced by a recorder -------------------

@pytest.fixture
def calls(monkeypatch):
    got = []
    monkeypatch.setattr(device, "_on_gpu", lambda *a: None)
    monkeypatch.setattr(device, "_other", lambda *a: None)
    monkeypatch.setattr(device, "_stream", lambda dev, st: 0 if st is None else st)
    monkeypatch.setattr(device, "_current_device", lambda: -1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    for name, value in (("moe_cache_write", None), ("moe_cache_read", None), ("moe_attention", None),
                        ("moe_attention_workspace_bytes", 1024), ("moe_attention_workspace_init", None)):
        monkeypatch.setattr(moe, name, lambda *a, name=name, value=value: got.append((name, a)) or value)
    return got


BF = torch.bfloat16
Z = torch.zeros


def a_cache(dtype=BF, **kw):
    quant = dtype == torch.float8_e4m3fn
    s = [Z(4, 2, 16).transpose(1, 2) for _ in range(2)] if quant else [None, None]
    args = dict(k=Z(4, 2, 16, 64, dtype=dtype).transpose(1, 2), v=Z(4, 2, 16, 64, dtype=dtype).transpose(1, 2),
                k_scale=s[0], v_scale=s[1])
    return device.PagedCache(**{**args, **kw})


def some_seqs(**kw):
    args = dict(starts=Z(3, dtype=torch.int32), kv_lens=Z(2, dtype=torch.int32), page_table=Z(2, 5, dtype=torch.int32))
    return device.Sequences(**{**args, **kw})


def refused(word, fn, *args, **kw):
    with pytest.raises(moe.MoEError) as e:
        fn(*args, **kw)
    assert e.value.code == ARG and word in str(e.value)


def test_caches_and_sequences_refuse(calls):
    a_cache(), a_cache(torch.float8_e4m3fn), some_seqs()
    for kw, word in ((dict(v=Z(4, 16, 2, 64)), "type"), (dict(v=Z(4, 16, 2, 48, dtype=BF)), "shape"),
                     (dict(v=Z(4, 16, 2, 64, dtype=BF)), "strides"), (dict(k=Z(4, 16, 64, dtype=BF)), "shape"),
                     (dict(k=Z(4, 16, 2, 64), v=Z(4, 16, 2, 64)), "float32"), (dict(k_scale=Z(4, 16, 2)), "no scales"),
                     (dict(k=Z(4, 16, 64, 2, dtype=BF).transpose(2, 3), v=Z(4, 16, 64, 2, dtype=BF).transpose(2, 3)), "contiguous")):
        refused(word, a_cache, **kw)
    for kw in (dict(k_scale=None), dict(v_scale=Z(4, 16, 3)), dict(k_scale=Z(4, 16, 2, dtype=BF)), dict(k_scale=Z(4, 16, 2))):
        refused("scale", a_cache, torch.float8_e4m3fn, **kw)
    for kw, word in ((dict(starts=Z(2, dtype=torch.int32)), "starts"), (dict(starts=Z(3)), "starts"), (dict(kv_lens=Z(2)), "kv_lens"),
                     (dict(page_table=Z(3, 5, dtype=torch.int32)), "page_table"), (dict(page_table=Z(5, dtype=torch.int32)), "page_table"),
                     (dict(page_table=Z(5, 2, dtype=torch.int32).t()), "contiguous"), (dict(max_rows=-1), "max_rows"),
                     (dict(starts=Z(6, dtype=torch.int32)[::2]), "contiguous")):
        refused(word, some_seqs, **kw)
    assert not calls


def test_moves_refuse_tensors(calls):
    c, s = a_cache(), some_seqs()
    ok = Z(3, 2, 64)
    for bad, word in ((Z(4, 2, 64), "shape"), (Z(3, 1, 64), "shape"), (Z(3, 2, 48), "shape"), (Z(3, 128), "shape"),
                      (Z(2, 3, 64).transpose(0, 1), "contiguous"), (Z(3, 64, 2).transpose(1, 2), "contiguous"), (Z(3, 2, 64, dtype=BF), "type")):
        refused(word, c.write, ok, bad, s)
        refused(word, c.read, s, k_out=ok, v_out=bad)
    refused("float64", c.write, ok.double(), ok.double(), s)
    refused("must be given", c.read, s)
    refused("must be given", c.read, s, rows=3, k_out=ok)
    assert not calls
    c.write(ok, ok, s)
    k, v = c.read(s, rows=7)
    assert k.shape == v.shape == (7, 2, 64) and k.dtype == BF
    assert [n for n, _ in calls] == ["moe_cache_write", "moe_cache_read"]
    assert calls[0][1][1]._obj.rows == 3 and calls[1][1][1]._obj.rows == 7


def test_attention_refuses_tensors(calls):
    c, s = a_cache(), some_seqs(max_rows=2)
    att = device.PagedAttention(4, 2, 64, device=_Cpu())
    del calls[:]
    q = Z(3, 4, 64, dtype=BF)
    for kw, word in ((dict(q=Z(3, 2, 64, dtype=BF)), "shape"), (dict(q=Z(3, 4, 48, dtype=BF)), "shape"), (dict(q=Z(3, 256, dtype=BF)), "shape"),
                     (dict(q=Z(4, 3, 64, dtype=BF).transpose(0, 1)), "contiguous"), (dict(q=Z(3, 4, 64, dtype=torch.float64)), "float64"),
                     (dict(out=Z(2, 4, 64, dtype=BF)), "shape"), (dict(out=Z(3, 4, 64)), "type"), (dict(lse=Z(3, 4, dtype=BF)), "lse"),
                     (dict(lse=Z(3, 5)), "lse"), (dict(lse=Z(4, 3).t()), "lse")):
        refused(word, att, **{**dict(q=q, cache=c, seqs=s), **kw})
    refused("heads", att, q, a_cache(k=Z(4, 16, 4, 64, dtype=BF), v=Z(4, 16, 4, 64, dtype=BF)), s)
    assert not calls
    out = att(q, c, s, lse=Z(3, 4))
    assert out.shape == q.shape and out.dtype == BF
    name, (a, cache, seqs, ws, ws_bytes, st) = calls[0]
    assert name == "moe_attention" and a.ld_q == a.ld_out == 256 and a.scale == 0.125 and seqs._obj.max_rows == 2 and seqs._obj.rows == 3


def test_moves_refuse_a_tensor_without_dimensions(calls):
    refused("shape", a_cache().write, Z(()), Z(3, 2, 64), some_seqs())
    refused("shape", a_cache().read, some_seqs(), k_out=Z(()), v_out=Z(()))
    assert not calls


@pytest.mark.parametrize("window", [-1, 1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 32) + 5])
def test_windows_that_32_bits_do_not_hold(calls, window):
    att = device.PagedAttention(4, 2, 64, device=_Cpu())
    del calls[:]
    q = Z(3, 4, 64, dtype=BF)
    refused("window", att, q, a_cache(), some_seqs(), window=window)
    assert not calls
    att(q, a_cache(), some_seqs(), window=0x7FFFFFFF)
    assert calls[0][1][0].window == 0x7FFFFFFF


class _Cpu:
    """Stands for a GPU: torch.device of the CPU with the index of its tensors."""


@pytest.fixture(autouse=True)
def _cpu_device(monkeypatch):
    real = torch.device

    class Dev:
        index = -1

    def fake(*a, **kw):
        return Dev() if a and isinstance(a[0], _Cpu) else real(*a, **kw)

    monkeypatch.setattr(device.torch, "device", fake)
    empty = torch.empty
    monkeypatch.setattr(device.torch, "empty", lambda *a, **kw: empty(*a, **{**kw, "device": "cpu"}) if isinstance(kw.get("device"), Dev)
                        else empty(*a, **kw))

"""Refusals of the operators in include/moe_block.h: arguments are checked on
the host before any launch, so these need no GPU."""
import ctypes

import pytest

from quantized_routed_expert_gemv_gb300 import build, moe


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


P = 1 << 20      # an aligned address; validation never reads through it


def norm_args(**kw):
    a = moe.moe_block_norm_args()
    a.y = a.h = a.h_out = a.x_out = a.w_post = a.w_pre = a.gate = P
    a.ld_y = a.ld_h = a.ld_h_out = a.ld_x_out = 64
    a.ld_gate_row, a.ld_gate_col = 0, 1
    a.rows, a.hidden, a.post_norm, a.pre_norm = 2, 64, 1, 1
    a.eps, a.residual_scale = 1e-6, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=-1), moe.MOE_ERR_ARG), (dict(hidden=0), moe.MOE_ERR_ARG), (dict(hidden=16385), moe.MOE_ERR_ARG),
    (dict(y=None, h=None), moe.MOE_ERR_ARG), (dict(h_out=None, x_out=None), moe.MOE_ERR_ARG),
    (dict(ld_y=63), moe.MOE_ERR_ARG), (dict(ld_h=0), moe.MOE_ERR_ARG), (dict(ld_h_out=1), moe.MOE_ERR_ARG),
    (dict(ld_x_out=-64), moe.MOE_ERR_ARG), (dict(y_type=3), moe.MOE_ERR_ARG), (dict(h_type=-1), moe.MOE_ERR_ARG),
    (dict(x_type=9), moe.MOE_ERR_ARG), (dict(w_type=5), moe.MOE_ERR_ARG), (dict(gate_type=4), moe.MOE_ERR_ARG),
    (dict(ld_gate_col=2), moe.MOE_ERR_ARG), (dict(ld_gate_row=-1), moe.MOE_ERR_ARG), (dict(eps=0.0), moe.MOE_ERR_ARG),
    (dict(eps=float("nan")), moe.MOE_ERR_ARG), (dict(w_add=0.5), moe.MOE_ERR_ARG), (dict(post_norm=2), moe.MOE_ERR_ARG),
    (dict(pre_norm=-1), moe.MOE_ERR_ARG), (dict(y=P + 1), moe.MOE_ERR_ALIGN),
    (dict(h=P + 2, h_type=moe.MOE_F32), moe.MOE_ERR_ALIGN), (dict(rows=0), moe.MOE_OK)])
def test_block_norm_refuses(L, kw, rc):
    a = norm_args(**kw)
    assert L.moe_block_norm(ctypes.byref(a), None) == rc
    if rc:
        assert "moe_block_norm" in moe.last_error()
    assert L.moe_block_norm(None, None) == moe.MOE_ERR_ARG


def lp_args(**kw):
    a = moe.moe_token_logprobs_args()
    a.logits = a.targets = a.target_logprobs = a.target_ranks = a.entropy = a.lse = a.top_ids = a.top_logprobs = P
    a.ld_logits, a.rows, a.vocab, a.n_targets, a.top_n, a.scale = 100, 2, 100, 1, 5, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=-1), moe.MOE_ERR_ARG), (dict(rows=(1 << 27) + 1), moe.MOE_ERR_ARG), (dict(vocab=0), moe.MOE_ERR_ARG),
    (dict(logits=None), moe.MOE_ERR_ARG), (dict(ld_logits=99), moe.MOE_ERR_ARG), (dict(logits_type=3), moe.MOE_ERR_ARG),
    (dict(n_targets=9), moe.MOE_ERR_ARG), (dict(n_targets=-1), moe.MOE_ERR_ARG), (dict(top_n=33), moe.MOE_ERR_ARG),
    (dict(top_n=-1), moe.MOE_ERR_ARG), (dict(targets=None), moe.MOE_ERR_ARG), (dict(scale=0.0), moe.MOE_ERR_ARG),
    (dict(scale=-1.0), moe.MOE_ERR_ARG), (dict(scale=float("inf")), moe.MOE_ERR_ARG),
    (dict(scale=float("nan")), moe.MOE_ERR_ARG), (dict(logits=P + 1), moe.MOE_ERR_ALIGN),
    (dict(lse=P + 2), moe.MOE_ERR_ALIGN), (dict(targets=P + 1), moe.MOE_ERR_ALIGN), (dict(rows=0), moe.MOE_OK)])
def test_token_logprobs_refuses(L, kw, rc):
    a = lp_args(**kw)
    assert L.moe_token_logprobs(ctypes.byref(a), None) == rc
    if rc:
        assert "moe_token_logprobs" in moe.last_error()
    assert L.moe_token_logprobs(None, None) == moe.MOE_ERR_ARG


def test_fp8_refuses(L):
    h = ctypes.c_void_p()
    ref = ctypes.byref(h)
    for n, k, codes, ld, scales, rc in [(0, 64, P, 64, P, moe.MOE_ERR_ARG), (64, 0, P, 64, P, moe.MOE_ERR_ARG),
                                        (64, 65537, P, 65552, P, moe.MOE_ERR_ARG), (64, 64, None, 64, P, moe.MOE_ERR_ARG),
                                        (64, 64, P, 64, None, moe.MOE_ERR_ARG), (64, 64, P, 63, P, moe.MOE_ERR_ARG),
                                        (64, 64, P, 72, P, moe.MOE_ERR_ARG), (64, 64, P + 8, 64, P, moe.MOE_ERR_ALIGN),
                                        (64, 64, P, 64, P + 2, moe.MOE_ERR_ALIGN)]:
        assert L.moe_fp8_open(n, k, codes, ld, scales, ref) == rc
        assert h.value is None and "moe_fp8_open" in moe.last_error()
    assert L.moe_fp8_open(64, 64, P, 64, P, None) == moe.MOE_ERR_ARG
    fake = (ctypes.c_uint8 * 4096)()   # zeroed host memory: wrong magic
    for w in (None, ctypes.addressof(fake)):
        assert L.moe_fp8_workspace_bytes(w, 1) == 0
        assert L.moe_fp8_workspace_init(w, P, 1 << 20, None) == moe.MOE_ERR_ARG
        assert L.moe_fp8_linear(w, P, 0, 64, 1, P, 0, 64, P, 1 << 20, None) == moe.MOE_ERR_ARG
        assert L.moe_fp8_check(w, P, None) == moe.MOE_ERR_ARG
        L.moe_fp8_close(w)             # ignored
    for args, rc in [((P, 0, 64, 0, 64, P, 64, P), moe.MOE_ERR_ARG), ((P, 3, 64, 64, 64, P, 64, P), moe.MOE_ERR_ARG),
                     ((None, 0, 64, 64, 64, P, 64, P), moe.MOE_ERR_ARG), ((P, 0, 63, 64, 64, P, 64, P), moe.MOE_ERR_ARG),
                     ((P, 0, 64, 64, 64, P, 72, P), moe.MOE_ERR_ARG), ((P + 1, 0, 64, 64, 64, P, 64, P), moe.MOE_ERR_ALIGN),
                     ((P, 0, 64, 64, 64, P + 4, 64, P), moe.MOE_ERR_ALIGN)]:
        assert L.moe_fp8_quantize_weights(*args, None) == rc, args

"""moe_block_norm against its formula in 64 bits.

Tolerance, derived: a thread adds at most 32 squares in sequence and the row
is joined in at most 10 further additions, so a mean square is within
42 * 2^-24 and its reciprocal root within half of that plus 2 ulp; with at
most six more roundings in a product, 2^-18 (64 * 2^-24) bounds the relative
error of each term.  h' = s h + g r may cancel, so its bound is relative to
|s h| + |g r|.  Storing adds half a unit of the output type: 2^-8 of the
value for bf16, 2^-11 for f16 (2^-25 absolute for its subnormals), 2^-24 for
f32."""
import pytest
import torch

from quantized_routed_expert_gemv_gb300 import moe
from quantized_routed_expert_gemv_gb300.device import block_norm

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ROUND = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}
ARITH = 2.0 ** -18


def formula(y, h, gate, w_post, w_pre, post_norm, pre_norm, w_add, eps, s):
    """(h', |s h| + |g r|, x, x's factor) in 64 bits."""
    like = h if h is not None else y
    H = like.shape[1]
    zero = torch.zeros(like.shape, dtype=torch.float64, device=like.device)
    r = zero if y is None else y.double()
    if post_norm:
        w = zero[0] if w_post is None else w_post.double()
        r = r / torch.sqrt((r * r).sum(1, keepdim=True) / H + eps) * (w + w_add)
    if gate is not None:
        r = r * gate.double()
    sh = zero if h is None else h.double() * s
    hn = sh + r
    f = torch.ones_like(hn)
    if pre_norm:
        w = zero[0] if w_pre is None else w_pre.double()
        f = (w + w_add) / torch.sqrt((hn * hn).sum(1, keepdim=True) / H + eps)
    return hn, sh.abs() + r.abs(), hn * f, f


def check(y, h, h_type=None, x_type=BF, gate=None, w_post=None, w_pre=None, post_norm=True, pre_norm=True, w_add=0.0,
          eps=1e-6, s=1.0, h_out=None, x_out=None):
    ref = formula(y, h, gate, w_post, w_pre, post_norm, pre_norm, w_add, eps, s)
    ho, xo = block_norm(y, h, gate=gate, w_post=w_post, w_pre=w_pre, post_norm=post_norm, pre_norm=pre_norm,
                        w_add=w_add, eps=eps, residual_scale=s, h_out=h_out, x_out=x_out, x_type=x_type)
    torch.cuda.synchronize()
    hn, mag, x, f = ref
    for got, want, terms in ((ho, hn, mag), (xo, x, mag * f.abs())):
        bound = ROUND[got.dtype] * want.abs() + ARITH * terms + 2.0 ** -25
        bad = (got.double() - want).abs() > bound
        assert not bad.any(), (got.dtype, bad.nonzero()[:3].tolist())
    return ho, xo


def rnd(*shape, dtype=BF, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


@pytest.mark.parametrize("H", [1, 2, 7, 8, 31, 33, 64, 250, 256, 257, 1000, 1999, 2048, 4097, 7168, 8192, 16383, 16384])
@pytest.mark.parametrize("T", [1, 3, 130])
def test_widths_and_rows(T, H):
    check(rnd(T, H, dtype=F32, seed=1), rnd(T, H, seed=2, scale=3.0), gate=rnd(H, seed=3), w_post=rnd(H, seed=4),
          w_pre=rnd(H, seed=5), w_add=1.0, s=0.75)


@pytest.mark.parametrize("yt", [BF, HF, F32])
@pytest.mark.parametrize("ht", [BF, HF, F32])
@pytest.mark.parametrize("xt", [BF, HF, F32])
@pytest.mark.parametrize("H", [512, 777])
def test_types(yt, ht, xt, H):
    wt = {BF: F32, HF: BF, F32: HF}[yt]
    check(rnd(9, H, dtype=yt, seed=1), rnd(9, H, dtype=ht, seed=2), x_type=xt, gate=rnd(9, H, dtype=xt, seed=3),
          w_post=rnd(H, dtype=wt, seed=4), w_pre=rnd(H, dtype=wt, seed=5), s=-1.5)


@pytest.mark.parametrize("shape", [(1, 640), (6, 1), (6, 640), (1, 1)])
@pytest.mark.parametrize("gt", [BF, F32])
def test_gates_broadcast(shape, gt):
    check(rnd(6, 640, seed=1), rnd(6, 640, seed=2), gate=rnd(*shape, dtype=gt, seed=3))


@pytest.mark.parametrize("pad_y,pad_h,pad_o", [(8, 8, 8), (1, 0, 8), (0, 3, 1), (5, 5, 5)])
@pytest.mark.parametrize("H", [640, 1021])
def test_strides(pad_y, pad_h, pad_o, H):
    T = 5
    y = rnd(T, H + pad_y, seed=1)[:, :H]
    h = rnd(T, H + pad_h, seed=2)[:, :H]
    guard = torch.full((T, H + pad_o), 7.0, dtype=BF, device=DEV)
    xo, ho = guard.clone(), guard.clone()
    gate = rnd(T, H + 3, seed=3)[:, :H]
    check(y, h, gate=gate, w_post=rnd(H, seed=4), w_pre=rnd(H, seed=5), h_out=ho[:, :H], x_out=xo[:, :H])
    if pad_o:
        assert (xo[:, H:] == 7.0).all() and (ho[:, H:] == 7.0).all()


def test_bases_off_sixteen_bytes():
    T, H = 4, 256
    buf = rnd(T * H + 3, seed=1)
    y = buf[3:].view(T, H)
    check(y, rnd(T, H, seed=2), w_post=rnd(H + 1, seed=3)[1:], w_pre=rnd(H + 1, seed=4)[1:])


@pytest.mark.parametrize("kw", [dict(post_norm=False), dict(pre_norm=False), dict(post_norm=False, pre_norm=False),
                                dict(w_add=1.0)])
def test_parts(kw):
    H = 2048
    y, h = rnd(3, H, dtype=F32, seed=1), rnd(3, H, seed=2)
    check(y, h, **kw)
    check(y, None, x_type=F32, w_post=rnd(H, seed=3), w_pre=rnd(H, seed=4), **kw)
    check(None, h, w_pre=rnd(H, seed=4), **kw)


@pytest.mark.parametrize("H", [257, 264, 1000, 2048, 4100, 7168, 8192, 9000])
@pytest.mark.parametrize("T", [1216, 2500])
def test_many_rows(T, H):
    """Enough rows for the streaming kernel, all in one pass and several per block."""
    pad = -H % 8
    y, h = rnd(T, H + pad, dtype=F32, seed=1)[:, :H], rnd(T, H + pad, seed=2)[:, :H]
    ho, xo = (torch.empty(T, H + pad, dtype=BF, device=DEV)[:, :H] for _ in range(2))
    check(y, h, gate=rnd(H, seed=3), w_post=rnd(H, seed=4), w_pre=rnd(H, seed=5), w_add=1.0, s=0.75, h_out=ho, x_out=xo)


@pytest.mark.parametrize("yt,ht,xt,wt", [(BF, BF, BF, F32), (F32, F32, F32, BF), (HF, BF, HF, HF), (BF, F32, BF, F32)])
@pytest.mark.parametrize("shape", [(1, 640), (1300, 1), (1300, 640)])
def test_many_rows_types_gates_and_parts(yt, ht, xt, wt, shape):
    T, H = 1300, 640
    y, h = rnd(T, H, dtype=yt, seed=1), rnd(T, H, dtype=ht, seed=2)
    w, v, g = rnd(H, dtype=wt, seed=4), rnd(H, dtype=wt, seed=5), rnd(*shape, dtype=xt, seed=3)
    for kw in (dict(), dict(post_norm=False), dict(pre_norm=False), dict(post_norm=False, pre_norm=False)):
        check(y, h, x_type=xt, gate=g, w_post=w, w_pre=v, **kw)
    check(y, None, x_type=xt, gate=g, w_post=w, w_pre=v)
    check(None, h, x_type=xt, w_pre=v)
    keep = h.clone()
    want = block_norm(y, h, gate=g, w_post=w, w_pre=v)
    _, x2 = block_norm(y, keep, gate=g, w_post=w, w_pre=v, h_out=keep)
    torch.cuda.synchronize()
    assert torch.equal(keep, want[0]) and torch.equal(x2, want[1])


def test_in_place_residual_and_repeat():
    T, H = 70, 7168
    y, h = rnd(T, H, dtype=F32, seed=1), rnd(T, H, seed=2)
    w, v = rnd(H, seed=3), rnd(H, seed=4)
    ho, xo = block_norm(y, h, w_post=w, w_pre=v, residual_scale=0.5)
    again = block_norm(y, h, w_post=w, w_pre=v, residual_scale=0.5)
    assert torch.equal(ho, again[0]) and torch.equal(xo, again[1])
    keep = h.clone()
    _, x2 = block_norm(y, keep, w_post=w, w_pre=v, residual_scale=0.5, h_out=keep)
    torch.cuda.synchronize()
    assert torch.equal(keep, ho) and torch.equal(x2, xo)


def test_zero_rows_and_special_values():
    H = 1024
    e = torch.empty(0, H, dtype=BF, device=DEV)
    ho, xo = block_norm(e, e)
    assert ho.shape == (0, H) and xo.shape == (0, H)
    # a row of zeros has the norm 0; NaN and infinities stay in their row
    y = rnd(4, H, dtype=F32, seed=1)
    h = rnd(4, H, seed=2)
    y[0], h[0] = 0.0, 0.0
    y[1, 5] = float("nan")
    h[2, 7] = float("inf")
    ho, xo = block_norm(y, h, w_add=1.0)
    torch.cuda.synchronize()
    assert (ho[0] == 0).all() and (xo[0] == 0).all()
    assert xo[1].isnan().all() and ho[1].isnan().all()
    assert ho[2, 7].isinf() and xo[2, 7].isnan() and (xo[2, :7] == 0).all()
    assert torch.isfinite(xo[3].float()).all()


def test_other_stream():
    H = 2048
    y, h = rnd(33, H, dtype=F32, seed=1), rnd(33, H, seed=2)
    want = block_norm(y, h, w_add=1.0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = block_norm(y, h, w_add=1.0, stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_refuses_on_the_gpu_box_too():
    y = rnd(2, 64)
    with pytest.raises(moe.MoEError) as e:
        block_norm(y, y, eps=0.0)
    assert e.value.code == moe.MOE_ERR_ARG

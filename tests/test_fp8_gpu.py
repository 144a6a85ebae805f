"""moe_fp8_linear against its definition in 64 bits.

The quantisation of x is exact arithmetic (powers of two) up to the rounding
to e4m3, so the reference below rounds the same values the same way and the
products are compared, not the quantisation's own error.

Tolerance, derived: a block's 128 products are exact in fp32 and summed in
the tensor core's fp32 accumulator; its order and truncation are not
documented, so a block sum is allowed 128 roundings of 2^-23 of the sum of its
products' magnitudes.  Scaling and adding ceil(K / 128) blocks rounds twice
each, 2^-24 of the running sum, at most of all magnitudes.  So
    |out - ref| <= (2^-16 + (2 blocks + 4) 2^-24) sum |x q| |w| + half a unit of
    the output type (2^-8, 2^-11 or 2^-24 of the value; 2^-25 for f16 subnormals)."""
import pytest
import torch

from quantized_routed_expert_gemv_gb300 import moe
from quantized_routed_expert_gemv_gb300.device import Fp8Linear

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ROUND = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}


def up(v, m):
    return -(-v // m) * m


def decode(codes):
    """e4m3 codes to float64 from their bit fields."""
    u = codes.to(torch.int64)
    e, m = (u >> 3) & 15, (u & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9)
    return torch.where(u >= 128, -v, v)


def quantised(x):
    """x's quantised values in float64."""
    T, K = x.shape
    p = torch.nn.functional.pad(x.double(), (0, up(K, 128) - K)).view(T, -1, 128)
    amax = p.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -200) / 448)).clamp(min=-126)
    s = torch.where(amax > 0, torch.exp2(e), torch.ones_like(amax))
    v = p / s
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step * s).view(T, -1)[:, :K]


def weights(n, k, seed=0, spread=True):
    """Codes (finite ones), scales and their float64 product."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ld = up(k, 16)
    codes = torch.randint(0, 256, (n, ld), generator=g, device=DEV, dtype=torch.int32)
    codes = torch.where((codes & 127) == 127, codes - 1, codes).to(torch.uint8)
    codes[:, k:] = 0x7F             # NaN codes in the padding take no part
    scales = torch.rand(-(-n // 128), -(-k // 128), generator=g, device=DEV) + 0.5
    if spread:
        scales *= torch.exp2(torch.randint(-6, 7, scales.shape, generator=g, device=DEV).float())
    w = decode(codes[:, :k]) * scales.double()[torch.arange(n, device=DEV) // 128][:, torch.arange(k, device=DEV) // 128]
    return codes, scales, w


def rnd(T, K, dtype=BF, seed=1, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, K + pad, generator=g, device=DEV) * torch.exp2(
        torch.randint(-4, 5, (T, 1), generator=g, device=DEV).float())
    return x.to(dtype)[:, :K]


def close(got, x, w, blocks):
    q = quantised(x)
    want, mag = q @ w.t(), q.abs() @ w.abs().t()
    bound = (2.0 ** -16 + (2 * blocks + 4) * 2.0 ** -24) * mag + ROUND[got.dtype] * want.abs() + 2.0 ** -25
    if got.dtype == HF:
        big = want.abs() + bound > 65504
        assert (got.double()[big].abs() > 60000).all()
        got, want, bound = got[~big], want[~big], bound[~big]
    bad = (got.double() - want).abs() > bound
    assert not bad.any(), ((got.double() - want).abs() / bound).max().item()


def check(T, N, K, xt=BF, ot=F32, pad=0, seed=0):
    codes, scales, w = weights(N, K, seed)
    lin = Fp8Linear(codes, scales, K, max_rows=T)
    x = rnd(T, K, xt, seed + 1, pad)
    guard = torch.full((T, N + pad), 7.0, dtype=ot, device=DEV)
    lin(x, guard[:, :N])
    torch.cuda.synchronize()
    assert lin.check() == moe.MOE_OK, moe.last_error()
    close(guard[:, :N], x, w, -(-K // 128))
    assert (guard[:, N:] == 7.0).all()
    lin.close()


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 100, 128, 129, 255, 256, 257, 500, 513])
def test_rows(T):
    check(T, 384, 512)


@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 1000, 2048, 20000])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_outputs(T, N):
    check(T, N, 256)


@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 127, 128, 129, 200, 1000, 1023, 2048, 7168])
@pytest.mark.parametrize("T", [1, 20, 150])
def test_inputs(T, K):
    check(T, 260, K, pad=3 if K % 2 else 0)


@pytest.mark.parametrize("xt", [BF, HF, F32])
@pytest.mark.parametrize("ot", [BF, HF, F32])
@pytest.mark.parametrize("T,pad", [(5, 0), (5, 1), (90, 8)])
def test_types_and_strides(xt, ot, T, pad):
    check(T, 700, 900, xt, ot, pad)


@pytest.mark.parametrize("T,N,K", [(4, 20000, 640), (130, 30000, 384), (1000, 5000, 1500), (700, 2048, 768),
                                   (300, 100, 7168), (16, 40000, 2048), (257, 40000, 300), (2000, 2100, 200),
                                   (777, 9999, 1111), (4000, 3000, 16)])
def test_many_tiles(T, N, K):
    check(T, N, K)


@pytest.mark.parametrize("xt,ot,pad", [(F32, BF, 0), (HF, HF, 3), (BF, BF, 8)])
def test_many_rows_types_and_strides(xt, ot, pad):
    check(1100, 4000, 700, xt, ot, pad)


def test_scales_of_x_at_their_edges():
    """Blocks whose largest value sits on, just above and just below 448 times a
    power of two, in the subnormals, at the type's largest, and blocks of zeros."""
    K = 128 * 10
    x = rnd(3, K, F32, 5)
    edge = [448.0, 448.0 * (1 + 2.0 ** -23), 448.0 * (1 - 2.0 ** -24), 2.0 ** -149, 2.0 ** -126, 1.0, 0.0, 3.0e38, 447.0, 2e-38]
    for b, m in enumerate(edge):
        blk = x[:, 128 * b:128 * b + 128]
        blk.copy_(blk.double().div(blk.double().abs().amax(1, keepdim=True)).mul(m).float())
        blk[:, 64] = m
    codes, scales, w = weights(256, K, 7, spread=False)
    codes2 = codes.clone()
    codes2[:, 7 * 128:8 * 128] = 0          # the block of 3e38 would hide the others
    lin, lin2 = Fp8Linear(codes, scales * 2.0 ** -20, K, 8), Fp8Linear(codes2, scales, K, 8)
    close(lin(x, out_type=F32), x, w * 2.0 ** -20, 10)
    w2 = w.clone()
    w2[:, 7 * 128:8 * 128] = 0
    close(lin2(x, out_type=F32), x, w2, 10)
    torch.cuda.synchronize()
    assert lin.check() == 0 and lin2.check() == 0


def test_single_products_are_exact():
    """One input and one weight: out is the product of the codes' values and
    the scales, exact in fp32."""
    codes = torch.arange(256, device=DEV).to(torch.uint8)
    codes = codes[(codes & 127) != 127]
    w = torch.zeros(codes.numel(), 16, dtype=torch.uint8, device=DEV)
    w[:, 0] = codes
    scales = torch.full((2, 1), 0.37, device=DEV)
    x = decode(codes).float()[:, None]
    lin = Fp8Linear(w, scales, 1, max_rows=300)
    out = lin(x, out_type=F32)
    torch.cuda.synchronize()
    close(out, x, decode(codes)[:, None] * scales[0, 0].double(), 1)
    q = quantised(x)
    assert torch.equal(out, (q.float() @ decode(codes).float()[None, :]) * scales[0, 0])


def test_nan_and_inf_rows():
    codes, scales, w = weights(300, 640, 3)
    x = rnd(20, 640, BF, 4)
    x[3, 600] = float("nan")
    x[7, 0] = float("inf")
    x[9, 10] = -float("inf")
    lin = Fp8Linear(codes, scales, 640, 20)
    out = lin(x, out_type=F32)
    torch.cuda.synchronize()
    bad = torch.zeros(20, dtype=torch.bool, device=DEV)
    bad[[3, 7, 9]] = True
    assert out[bad].isnan().all()
    close(out[~bad], x[~bad], w, 5)


def test_workspace_shared_repeat_and_stream():
    """Handles of other shapes take turns on one workspace; a call repeated,
    with other row counts between and on another stream, gives the same bits."""
    a = Fp8Linear(*weights(520, 1024, 1)[:2], 1024, 300)
    b = Fp8Linear(*weights(2000, 384, 2)[:2], 384, 300)
    b.ws_ptr, b.ws_bytes = a.ws_ptr, a.ws_bytes
    xa, xb = rnd(300, 1024), rnd(300, 384)
    first = a(xa, out_type=F32), b(xb, out_type=F32)
    for T in (1, 17, 33, 100, 200):
        # rows do not depend on their neighbours' values
        other = rnd(T, 1024, seed=T)
        other[0] = xa[0]
        same = a(other, out_type=F32)
        again = a(xa[:T], out_type=F32)
        assert torch.equal(same[0], again[0])
        b(xb[:T])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        second = a(xa, out_type=F32), b(xb, out_type=F32)
    st.synchronize()
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
    assert a.check() == 0


def test_graph_capture():
    lin = Fp8Linear(*weights(1000, 512, 1)[:2], 512, 64)
    x, out = rnd(64, 512), torch.empty(64, 1000, device=DEV)
    want = lin(x, out_type=F32).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin(x, out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("n,k", [(1, 1), (130, 300), (1000, 2048), (256, 128)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_quantised_weights(n, k, dtype):
    """Codes are the nearest e4m3 values of w / scale, scale = max |w| / 448 of
    each block; the padding is 0."""
    w = rnd(n, k + 3, dtype)[:, :k]
    if n > 200 and k > 128:
        w[128:256, :128] = 0
    lin = Fp8Linear.from_weights(w, 4)
    torch.cuda.synchronize()
    p = torch.zeros(up(n, 128), up(k, 128), device=DEV)
    p[:n, :k] = w.float()
    b = p.view(-1, 128, p.shape[1] // 128, 128)
    amax = b.abs().amax((1, 3))
    # a tensor as divisor: division by a Python number multiplies by its reciprocal on CUDA
    scales = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    assert torch.equal(lin.scales, scales)
    v = (b / scales[:, None, :, None]).view_as(p)[:n, :k]
    assert torch.equal(decode(lin.codes[:, :k]).float(), v.to(torch.float8_e4m3fn).float())
    assert (lin.codes[:, k:] == 0).all()
    x = rnd(4, k)
    close(lin(x, out_type=F32), x, decode(lin.codes[:, :k]) * scales.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k], -(-k // 128))


def test_refuses_and_empty():
    lin = Fp8Linear(*weights(200, 256, 1)[:2], 256, 16)
    assert lin(rnd(0, 256)).shape == (0, 200)
    with pytest.raises(moe.MoEError) as e:
        lin(rnd(17, 256))               # the workspace is too small
    assert e.value.code == moe.MOE_ERR_ARG and "workspace" in str(e.value)
    with pytest.raises(moe.MoEError) as e:
        moe.moe_fp8_linear(lin.handle, lin.codes.data_ptr(), moe.MOE_BF16, 255, 1, lin.codes.data_ptr(), moe.MOE_BF16,
                           200, lin.ws_ptr, lin.ws_bytes)
    assert e.value.code == moe.MOE_ERR_ARG
    with pytest.raises(moe.MoEError) as e:
        moe.moe_fp8_linear(lin.handle, lin.codes.data_ptr() + 1, moe.MOE_BF16, 256, 1, lin.codes.data_ptr(),
                           moe.MOE_BF16, 200, lin.ws_ptr, lin.ws_bytes)
    assert e.value.code == moe.MOE_ERR_ALIGN
    lin.close()
    with pytest.raises(moe.MoEError):
        lin.handle = None
        lin(rnd(1, 256))

"""What the tensor wrappers of device.py refuse before the library, which sees
addresses only, could read or write past a tensor.  The library is replaced by
a recorder, so nothing runs and no GPU is needed; tensors of the CPU stand for a
GPU's except where that is what is refused."""
import pytest
import torch

from quantized_routed_expert_gemv_gb300 import device, moe

BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """The names of the library calls that a wrapper got through to."""
    got = []
    monkeypatch.setattr(device, "_on_gpu", lambda *a: None)
    monkeypatch.setattr(device, "_other", lambda *a: None, raising=False)

    def record(name, value=None):
        monkeypatch.setattr(moe, name, lambda *a: got.append(name) or value)

    record("moe_block_norm"), record("moe_token_logprobs"), record("moe_fp8_linear")
    record("moe_fp8_open", 0), record("moe_fp8_workspace_bytes", 512), record("moe_fp8_workspace_init")
    record("moe_fp8_quantize_weights"), record("moe_fp8_close")
    return got


def refused(calls, word, fn, *args, **kw):
    del calls[:]
    with pytest.raises(moe.MoEError) as e:
        fn(*args, stream=0, **kw)
    assert e.value.code == moe.MOE_ERR_ARG and word in str(e.value)
    assert not calls


def m(rows, cols, dtype=BF):
    return torch.zeros(rows, cols, dtype=dtype)


@pytest.mark.parametrize("kw,word", [
    (dict(y=m(3, 64)), "y"), (dict(y=m(5, 64)), "y"), (dict(y=m(4, 63)), "y"), (dict(y=m(4, 65)), "y"),
    (dict(y=torch.zeros(4 * 64)), "y"), (dict(h_out=m(3, 64)), "h_out"), (dict(h_out=m(4, 32)), "h_out"),
    (dict(x_out=m(3, 64)), "x_out"), (dict(x_out=m(4, 128)), "x_out"), (dict(w_post=torch.zeros(63)), "w_post"),
    (dict(w_pre=torch.zeros(1, 64)), "w_pre"), (dict(w_pre=torch.zeros(128)[::2]), "w_pre"),
    (dict(w_post=torch.zeros(64), w_pre=torch.zeros(64, dtype=BF)), "w_pre"), (dict(gate=torch.zeros(3, 64)), "gate"),
    (dict(gate=torch.zeros(4, 32)), "gate"), (dict(h_out=m(4, 64, torch.float32)), "h_out"),
    (dict(y=m(4, 64, torch.float64)), "float64"), (dict(x_type=torch.int32), "int32"), (dict(y=m(64, 4).t()), "contiguous"),
    (dict(h=torch.zeros(4, 2, 32)), "matrix"), (dict(h=None, y=None), "matrix")])
def test_block_norm(calls, kw, word):
    refused(calls, word, device.block_norm, **{**dict(y=m(4, 64), h=m(4, 64)), **kw})


@pytest.mark.parametrize("kw,word", [
    (dict(targets=torch.zeros(3, dtype=torch.int32)), "targets"), (dict(targets=torch.zeros(4, dtype=torch.int64)), "targets"),
    (dict(targets=torch.zeros(4, 4, dtype=torch.int32).t()[:, ::2]), "targets"),
    (dict(targets=torch.tensor(3, dtype=torch.int32)), "targets"), (dict(logits=torch.zeros(4 * 100)), "matrix"),
    (dict(logits=m(100, 4).t()), "contiguous"), (dict(logits=m(4, 100, torch.float64)), "float64")])
def test_token_logprobs(calls, kw, word):
    refused(calls, word, device.token_logprobs, **{**dict(logits=m(4, 100)), **kw})


@pytest.mark.parametrize("kw,word", [
    (dict(codes=torch.zeros(200, 96, dtype=torch.uint8)), "codes"), (dict(codes=torch.zeros(200, 112)), "codes"),
    (dict(codes=torch.zeros(200 * 112, dtype=torch.uint8)), "codes"), (dict(scales=torch.zeros(1, 1)), "scales"),
    (dict(scales=torch.zeros(2, 1, dtype=BF)), "scales"), (dict(scales=torch.zeros(2, 2)[:, :1]), "scales")])
def test_fp8_weights(calls, kw, word):
    args = {**dict(codes=torch.zeros(200, 112, dtype=torch.uint8), scales=torch.zeros(2, 1)), **kw}
    refused(calls, word, device.Fp8Linear, args["codes"], args["scales"], 100, 8)
    refused(calls, "matrix", device.Fp8Linear.from_weights, torch.zeros(5), 8)
    refused(calls, "float64", device.Fp8Linear.from_weights, m(5, 5, torch.float64), 8)


@pytest.mark.parametrize("x,out,word", [
    (m(4, 99), None, "x"), (m(4, 101), None, "x"), (torch.zeros(100), None, "x"), (m(4, 100), m(3, 200), "out"),
    (m(4, 100), m(4, 199), "out"), (m(4, 100), m(200, 4).t(), "contiguous"), (m(4, 100), m(4, 200, torch.float64), "float64"),
    (m(4, 100, torch.int8), None, "int8")])
def test_fp8_linear(calls, x, out, word):
    lin = device.Fp8Linear(torch.zeros(200, 112, dtype=torch.uint8), torch.zeros(2, 1), 100, 8, stream=0)
    refused(calls, word, lin, x, out)


def test_tensors_of_the_cpu(calls, monkeypatch):
    lin = device.Fp8Linear(torch.zeros(200, 112, dtype=torch.uint8), torch.zeros(2, 1), 100, 8, stream=0)
    monkeypatch.undo()
    for name in ("moe_block_norm", "moe_token_logprobs", "moe_fp8_linear", "moe_fp8_open", "moe_fp8_quantize_weights"):
        monkeypatch.setattr(moe, name, lambda *a, name=name: calls.append(name))
    lin.index = 0
    refused(calls, "cpu", device.block_norm, m(4, 64), m(4, 64))
    refused(calls, "cpu", device.token_logprobs, m(4, 100))
    refused(calls, "cpu", device.Fp8Linear, lin.codes, lin.scales, 100, 8)
    refused(calls, "cpu", device.Fp8Linear.from_weights, m(4, 64), 8)
    refused(calls, "cpu", lin, m(4, 100), m(4, 200))


@pytest.mark.gpu
def test_one_tensor_of_the_cpu(calls, monkeypatch):
    c = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype, device="cuda:0")  # noqa: E731
    lin = device.Fp8Linear(c(200, 112, dtype=torch.uint8), c(2, 1, dtype=torch.float32), 100, 8, stream=0)
    monkeypatch.undo()
    for name in ("moe_block_norm", "moe_token_logprobs", "moe_fp8_linear", "moe_fp8_open"):
        monkeypatch.setattr(moe, name, lambda *a, name=name: calls.append(name))
    lin.index = 0
    for kw in (dict(y=m(4, 64)), dict(h=m(4, 64)), dict(gate=m(1, 64)), dict(w_post=m(1, 64)[0]), dict(w_pre=m(1, 64)[0]),
               dict(h_out=m(4, 64)), dict(x_out=m(4, 64))):
        refused(calls, "cpu", device.block_norm, **{**dict(y=c(4, 64), h=c(4, 64)), **kw})
    refused(calls, "cpu", device.token_logprobs, c(4, 100), torch.zeros(4, dtype=torch.int32))
    refused(calls, "cpu", device.Fp8Linear, lin.codes, lin.scales.cpu(), 100, 8)
    refused(calls, "cpu", lin, m(4, 100), c(4, 200))
    refused(calls, "cpu", lin, c(4, 100), m(4, 200))

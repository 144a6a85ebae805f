"""Calls of the tensor wrappers on another stream than torch's current one: what
they allocate is that stream's memory, and in use on the current one too."""
import pytest
import torch

from quantized_routed_expert_gemv_gb300 import device, moe
from quantized_routed_expert_gemv_gb300.device import Fp8Linear, block_norm, token_logprobs

BF = torch.bfloat16


def test_outputs_are_allocated_on_the_given_stream(monkeypatch):
    """With the library, the streams and the GPU replaced by recorders."""
    now, seen, used = [7], [], []

    class Other:
        def __init__(self, raw, dev):
            self.raw = raw

    class Use:
        def __init__(self, st):
            self.st = st

        def __enter__(self):
            now.append(self.st.raw)

        def __exit__(self, *a):
            now.pop()

    plain = torch.empty

    def empty(*a, **kw):
        seen.append(now[-1])
        return plain(*a, **kw)

    monkeypatch.setattr(torch.cuda, "ExternalStream", Other)
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Other(now[-1], dev))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, st: used.append(st.raw))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(device, "_stream", lambda dev, st: 7 if st is None else st)
    monkeypatch.setattr(device, "_on_gpu", lambda *a: None, raising=False)
    for name in ("block_norm", "token_logprobs", "fp8_linear", "fp8_workspace_init", "fp8_quantize_weights", "fp8_close"):
        monkeypatch.setattr(moe, "moe_" + name, lambda *a: None)
    monkeypatch.setattr(moe, "moe_fp8_open", lambda *a: 0)
    monkeypatch.setattr(moe, "moe_fp8_workspace_bytes", lambda *a: 256)
    z = torch.zeros
    for given, want in ((9, 9), (7, 7), (None, 7), (0, 0)):
        del seen[:], used[:]
        block_norm(z(4, 64), z(4, 64), stream=given)
        assert seen == [want] * 2 and used == ([7] * 2 if want != 7 else [])
        del seen[:], used[:]
        token_logprobs(z(4, 100), z(4, dtype=torch.int32), top_n=3, stream=given)
        assert seen == [want] * 6 and used == ([7] * 6 if want != 7 else [])
        del seen[:], used[:]
        lin = Fp8Linear.from_weights(z(200, 100), 8, stream=given)
        assert seen == [want] * 3 and used == ([7] * 3 if want != 7 else [])
        del seen[:], used[:]
        lin(z(4, 100), stream=given)
        assert seen == [want]
        # the layer's own tensors are in use on the call's stream, the output on the current one
        assert used == ([want] * 3 + [7] if want != 7 else [])
        del seen[:]
        lin(z(4, 100), plain(4, 200), stream=given)
        assert seen == []


@pytest.mark.gpu
def test_freed_memory_with_work_in_flight():
    """Memory freed while the current stream still has to read it is not what a
    call on another stream writes."""
    dev = "cuda:0"
    y = torch.randn(64, 2048, device=dev)
    lin = Fp8Linear.from_weights(torch.randn(2048, 2048, device=dev), 64)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda: block_norm(y, y, x_type=torch.float32, stream=other.cuda_stream),
                 lambda: lin(y, out_type=torch.float32, stream=other.cuda_stream),
                 lambda: token_logprobs(y, top_n=32, stream=other.cuda_stream)):
        call()                                  # the other stream's memory is there
        torch.cuda.synchronize()
        a = [torch.full((64, 2048), 7.0, device=dev) for _ in range(4)] + [torch.full((64, 32), 7.0, device=dev)]
        at = {t.data_ptr() for t in a}
        torch.cuda._sleep(20_000_000)           # about 10 ms, then the copies
        kept = [t.clone() for t in a]
        del a
        out = call()
        outs = list(out.values()) if isinstance(out, dict) else list(out) if isinstance(out, tuple) else [out]
        assert not {t.data_ptr() for t in outs} & at
        torch.cuda.synchronize()
        assert all((t == 7.0).all() for t in kept)


@pytest.mark.gpu
def test_results_on_other_streams():
    dev = "cuda:0"
    y, w = torch.randn(33, 1000, device=dev), torch.randn(500, 1000, device=dev)
    lin = Fp8Linear.from_weights(w, 64)
    want = block_norm(y, y), lin(y), token_logprobs(y, top_n=3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    # on a side stream; and, with a side stream current, on the default one (raw handle 0)
    for current, raw in ((torch.cuda.current_stream(), side.cuda_stream), (side, torch.cuda.default_stream().cuda_stream)):
        with torch.cuda.stream(current):
            lin2 = Fp8Linear.from_weights(w, 64, stream=raw)
            got = block_norm(y, y, stream=raw), lin(y, stream=raw), token_logprobs(y, top_n=3, stream=raw), lin2(y, stream=raw)
            torch.cuda.synchronize()
        assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][1], want[0][1])
        assert torch.equal(got[1], want[1]) and torch.equal(got[3], want[1])
        for k in want[2]:
            assert torch.equal(got[2][k], want[2][k])

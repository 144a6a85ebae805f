"""examples/score_tokens.py: the operators around the layer run together.

Each operator's outputs are compared with plain arithmetic in 64 bits on the
operator's own inputs of that run, with the tolerances of its own test file
(half a unit of bf16 plus 2^-18 of the terms for the boundary; 2^-16 of the
magnitudes for the product), and decoding agrees with scoring what was
decoded."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("score_tokens", os.path.join(ROOT, "examples", "score_tokens.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rms(v):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)


def test_each_operator_in_the_run(example):
    from test_fp8_gpu import close, decode
    stack = example.Stack()
    tokens = torch.arange(5, 5 + 33 * 11, 11, device="cuda:0")
    trace = []
    logits = stack.logits(tokens, trace)
    out = example.token_logprobs(logits, torch.roll(tokens, -1).to(torch.int32), top_n=4)
    torch.cuda.synchronize()
    stack.check()
    for i, (y, h, h2, x) in enumerate(trace[:-1]):
        r = rms(y.double()) * (1 + stack.w_post[i].double()) * stack.gate[i].double()
        want = h.double() * 0.9 + r
        mag = h.double().abs() * 0.9 + r.abs()
        assert ((h2.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * mag).all()
        f = (1 + stack.w_pre[i + 1].double()) / torch.sqrt((want * want).mean(1, keepdim=True) + 1e-6)
        assert ((x.double() - want * f).abs() <= 2.0 ** -8 * (want * f).abs() + 2.0 ** -18 * mag * f.abs()).all()
    x, got = trace[-1]
    n, k = stack.head.n, stack.head.k
    s = stack.head.scales.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    close(got, x, decode(stack.head.codes[:, :k]) * s, -(-k // 128))
    lp = torch.log_softmax(logits.double(), 1)
    want = lp.gather(1, torch.roll(tokens, -1)[:, None])[:, 0]
    assert ((out["logprob"].double() - want).abs() <= 1e-5).all()
    assert torch.equal(out["top_ids"][:, 0].long(), logits.argmax(1))
    assert ((out["entropy"].double() + (lp.exp() * lp).sum(1)).abs() <= 1e-4).all()
    stack.close()


def test_decoding_agrees_with_scoring(example):
    """The log probabilities of decoded tokens equal those of the same tokens
    scored as a prompt (one chunk, the other paths of layer and product), to
    the layer's own 2e-3 and the head's bf16 input."""
    stack = example.Stack()
    start = torch.tensor([17], device="cuda:0")
    ids, logprobs = example.decode(stack, start, 20)
    s = example.score(stack, torch.cat([start, ids]))
    torch.cuda.synchronize()
    stack.check()
    assert (s["rank"] <= 2).all()
    assert ((s["logprob"] - logprobs).abs() <= 0.1).all()
    stack.close()


def test_main_prints(example, capsys):
    example.main()
    text = capsys.readouterr().out
    assert "prompt of 40 tokens" in text and "decoded:" in text

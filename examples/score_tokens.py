"""Scores a prompt and decodes a few tokens through a stack of Mixture-of-Experts
layers: the operators of include/moe_block.h and include/moe_fp8.h around the
layer of include/moe.h, as a serving loop would call them.

    h = embedding[token]
    x = norm(h)                                   moe_block_norm (pre-norm only)
    for every layer:
        y    = layer(x)                           moe_prefill_chunk / moe_decode
        h, x = boundary(y, h)                     moe_block_norm (post-norm, gate,
                                                  scaled residual, next pre-norm)
    logits = head(x)                              moe_fp8_linear
    log probabilities, ranks, alternatives        moe_token_logprobs

The stack has no attention and random weights: every token depends on its
predecessor alone.  Run on a GB300 after building:

    python examples/score_tokens.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_routed_expert_gemv_gb300 import moe, synth  # noqa: E402
from quantized_routed_expert_gemv_gb300.device import DeviceLayer, Fp8Linear, block_norm, token_logprobs  # noqa: E402


class Stack:
    def __init__(self, shape=synth.TINY, layers: int = 2, vocab: int = 1000, max_tokens: int = 128, seed: int = 7,
                 device="cuda:0"):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device=device) * scale).to(torch.bfloat16)  # noqa: E731
        H = shape.H
        self.embedding = rnd(vocab, H)
        self.layers = [DeviceLayer(shape, seed, layer=i, max_tokens=max_tokens, device=device) for i in range(layers)]
        # weights of the norms as their distance from one, a gate for every channel
        self.w_pre = [rnd(H, scale=0.1) for _ in range(layers + 1)]
        self.w_post = [rnd(H, scale=0.1) for _ in range(layers)]
        self.gate = [rnd(H, scale=0.1) + 0.5 for _ in range(layers)]
        self.residual_scale = 0.9
        self.head = Fp8Linear.from_weights(rnd(vocab, H, scale=H ** -0.5), max_rows=max_tokens)

    def logits(self, tokens: torch.Tensor, trace=None) -> torch.Tensor:
        """float32 logits [rows][vocab] after each of the tokens (device int64)."""
        h = self.embedding[tokens]
        _, x = block_norm(h=h, w_pre=self.w_pre[0], post_norm=False, w_add=1.0)
        for i, layer in enumerate(self.layers):
            # the tensor-core path for a chunk, the few-token path for a decode step
            _, y, _, _ = (layer.prefill if len(tokens) > 16 else layer.decode)(x)
            before = h.clone() if trace is not None else None
            # the residual stream is updated in place; x feeds the next layer
            h, x = block_norm(y, h, gate=self.gate[i], w_post=self.w_post[i], w_pre=self.w_pre[i + 1], w_add=1.0,
                              residual_scale=self.residual_scale, h_out=h)
            if trace is not None:
                trace.append((y, before, h.clone(), x))
        out = self.head(x, out_type=torch.float32)
        if trace is not None:
            trace.append((x, out))
        return out

    def check(self) -> None:
        """Raises if device code latched an error."""
        for status in [layer.check() for layer in self.layers] + [self.head.check()]:
            if status != moe.MOE_OK:
                raise RuntimeError(moe.last_error())

    def close(self) -> None:
        for layer in self.layers:
            layer.close()
        self.head.close()


def score(stack: Stack, tokens: torch.Tensor, top_n: int = 3) -> dict:
    """Log probability and rank of every token after the first, the entropy in
    its place, and the likeliest tokens after the last."""
    out = token_logprobs(stack.logits(tokens), torch.roll(tokens, -1).to(torch.int32), top_n=top_n)
    return {"logprob": out["logprob"][:-1], "rank": out["rank"][:-1], "entropy": out["entropy"][:-1],
            "next_ids": out["top_ids"][-1], "next_logprobs": out["top_logprobs"][-1]}


def decode(stack: Stack, token: torch.Tensor, steps: int):
    """Greedy decoding from one token (device int64 [1]): ids and log probabilities."""
    ids, logprobs = [], []
    for _ in range(steps):
        out = token_logprobs(stack.logits(token), top_n=1)
        token = out["top_ids"][:, 0].long()
        ids.append(token)
        logprobs.append(out["top_logprobs"][:, 0])
    return torch.cat(ids), torch.cat(logprobs)


def main() -> None:
    stack = Stack()
    prompt = torch.arange(3, 3 + 40 * 17, 17, device="cuda:0")
    s = score(stack, prompt)
    ids, logprobs = decode(stack, prompt[-1:], 8)
    torch.cuda.synchronize()
    stack.check()
    print("prompt of %d tokens: log probability %.3f, mean entropy %.3f, median rank %d" % (
        len(prompt), s["logprob"].sum().item(), s["entropy"].mean().item(), s["rank"].median().item()))
    print("next:", ", ".join("%d (%.3f)" % p for p in zip(s["next_ids"].tolist(), s["next_logprobs"].tolist())))
    print("decoded:", ", ".join("%d (%.3f)" % p for p in zip(ids.tolist(), logprobs.tolist())))
    stack.close()


if __name__ == "__main__":
    main()

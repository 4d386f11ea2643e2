"""Greedy decoding through one block on 4-bit weights: a projection, a mixture
of experts, the head, and the log probabilities of what they answer.

    python examples/decode_step.py --fmt mxfp4 --batch 4 --steps 16

The weights are random.  Every layer is quantized by the library (the weight
side of its transform first, where it has one) and multiplied by linear_w4 or
moe_w4 (the activation side online); token_logprobs scores the next token and
names the alternatives.  Attention and norms are not part of it.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_activation_amd as wush  # noqa: E402
from mxfp4_activation_amd import layerwise, transforms  # noqa: E402

GROUP = {"mxfp4": 32, "nvfp4": 16, "int4": 32}


class Block:
    """Projection with its own WUSH transforms, experts with blockwise Hadamard
    transforms, a head without any."""

    def __init__(self, fmt: str, vocab: int, hidden: int, experts: int, top_k: int, inner: int, seed: int = 0):
        G, dev = GROUP[fmt], torch.device("cuda")
        gen = torch.Generator(device=dev).manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen, device=dev) * std).to(torch.bfloat16)

        self.fmt, self.top_k = fmt, top_k
        self.embed = normal(vocab, hidden)
        self.router = normal(experts, hidden, std=hidden**-0.5)
        proj = normal(hidden, hidden, std=hidden**-0.5)
        self.proj_T, weight_T, _, _ = transforms.wush_bank(proj, self.embed[: 4 * hidden].contiguous(), G)
        self.proj = layerwise.quantize(fmt, proj, weight_T)
        self.head = layerwise.quantize(fmt, normal(vocab, hidden, std=hidden**-0.5),
                                       transforms.identity_bank(hidden // G, G, dev))
        t_in, t_mid = (transforms.hadamard_bank(n // G, G, dev) for n in (hidden, inner))
        self.gate_up = self._experts([normal(2 * inner, hidden, std=hidden**-0.5) for _ in range(experts)], t_in, t_in)
        self.down = self._experts([normal(hidden, inner, std=inner**-0.5) for _ in range(experts)], t_mid,
                                  t_mid.repeat(experts, 1, 1, 1))

    def _experts(self, weights, weight_T, T) -> wush.W4Experts:
        parts = [layerwise.quantize(self.fmt, w, weight_T) for w in weights]
        scale = torch.cat([p[2].reshape(1) for p in parts]) if self.fmt == "nvfp4" else None
        return wush.W4Experts(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]), scale, T)

    def logits(self, tokens: torch.Tensor):
        """fp32 logits of the tokens after `tokens` [M], and the experts' choice."""
        x = self.embed[tokens]
        codes, scales, g = self.proj
        x = x + wush.linear_w4(self.fmt, x, codes, scales, T=self.proj_T, global_scale=g)
        moe = wush.moe_w4(self.fmt, x, self.router, self.gate_up, self.down, self.top_k)
        codes, scales, g = self.head
        return wush.linear_w4(self.fmt, x + moe.out, codes, scales, global_scale=g, out_dtype=torch.float32), moe


def decode(block: Block, tokens: torch.Tensor, steps: int, top: int = 5):
    """Greedy continuation of tokens [M]: (tokens [steps, M], their log
    probabilities and the entropies, both [steps, M])."""
    nothing = torch.full_like(tokens, -1)
    ids, logprobs, entropies = [], [], []
    for _ in range(steps):
        logits, _ = block.logits(tokens)
        answer = wush.token_logprobs(logits, nothing, top=top)
        tokens = answer.top_ids[:, 0].long()
        ids.append(tokens)
        logprobs.append(answer.top_logprobs[:, 0])
        entropies.append(answer.entropy)
    return torch.stack(ids), torch.stack(logprobs), torch.stack(entropies)


def score(block: Block, text: torch.Tensor) -> torch.Tensor:
    """Log probabilities of text [n + 1]'s tokens after the first, each from the one before."""
    logits, _ = block.logits(text[:-1])
    return wush.token_logprobs(logits, text[1:].contiguous()).logprob


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--fmt", choices=sorted(GROUP), default="mxfp4")
    p.add_argument("--vocab", type=int, default=32768)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--inner", type=int, default=1024)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--top-k", type=int, default=4)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--steps", type=int, default=16)
    a = p.parse_args(argv)
    block = Block(a.fmt, a.vocab, a.hidden, a.experts, a.top_k, a.inner)
    first = torch.arange(a.batch, device="cuda")
    decode(block, first, 2)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    ids, logprobs, entropies = decode(block, first, a.steps)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) * 1e3 / a.steps
    text = torch.cat([first[:1], ids[:, 0]])
    print("%s, %d sequences: %.3f ms a step; mean log probability %.4f, entropy %.4f; perplexity of the first %.4f"
          % (a.fmt, a.batch, ms, logprobs.mean(), entropies.mean(), float(torch.exp(-score(block, text).mean()))))
    return ids, logprobs, entropies


if __name__ == "__main__":
    main()

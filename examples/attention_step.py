"""Greedy decoding of several requests through an attention block in 4 bits: a
fused query, key and value projection with every request's own low-rank adapter, a
paged cache of keys and values in 4 bits, attention over it, the output projection,
the head, penalties for repeated tokens, and the log probabilities of what they answer.

    python examples/attention_step.py --fmt mxfp4 --requests 4 --prompt 500 --steps 16

The weights are random; positions and norms are not part of it.  Keys go through
blockwise Hadamard transforms on their way into the cache, and the queries through the
same ones; values are kept in a Hadamard basis, which the output projection's
weights take as it is (they were quantized with the weight side of that transform).
"""

from __future__ import annotations

import argparse
import os
import sys
import time
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_activation_amd as wush  # noqa: E402
from mxfp4_activation_amd import layerwise, transforms  # noqa: E402

GROUP = {"mxfp4": 32, "nvfp4": 16, "int4": 32}


class Step(NamedTuple):
    """What one pass computes on its way, for those who want to look."""
    x: torch.Tensor
    qkv: torch.Tensor
    attention: torch.Tensor
    hidden: torch.Tensor
    logits: torch.Tensor


class Block:
    def __init__(self, fmt: str, vocab: int, hidden: int, q_heads: int, heads: int, D: int, adapters: int, rank: int,
                 seed: int = 0):
        G, dev = GROUP[fmt], torch.device("cuda")
        gen = torch.Generator(device=dev).manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen, device=dev) * std).to(torch.bfloat16)

        self.fmt, self.q_heads, self.heads, self.D = fmt, q_heads, heads, D
        rows = (q_heads + 2 * heads) * D
        self.embed = normal(vocab, hidden)
        qkv = normal(rows, hidden, std=hidden**-0.5)
        self.qkv_T, weight_T, _, _ = transforms.wush_bank(qkv, self.embed[: 4 * hidden].contiguous(), G)
        self.qkv = layerwise.quantize(fmt, qkv, weight_T)
        self.adapters = wush.LoraAdapters(normal(adapters, rank, hidden, std=hidden**-0.5),
                                          normal(adapters, rows, rank, std=rank**-0.5), torch.full((adapters,), 0.2, device=dev))
        self.cache_T = transforms.hadamard_bank(D // G, G, dev).repeat(heads, 1, 1, 1)
        self.out = layerwise.quantize(fmt, normal(hidden, q_heads * D, std=(q_heads * D) ** -0.5),
                                      transforms.hadamard_bank(q_heads * D // G, G, dev))
        self.head = layerwise.quantize(fmt, normal(vocab, hidden, std=hidden**-0.5),
                                       transforms.identity_bank(hidden // G, G, dev))

    def cache(self, pages: int, page: int) -> wush.KV4Cache:
        # Calibrated tensor scales: normal keys and values stay below 8.
        g = torch.full((1,), 8.0 / 2688, device="cuda") if self.fmt == "nvfp4" else None
        return wush.kv4_cache(self.fmt, pages, self.heads, page, self.D, k_global=g, v_global=g)

    def step(self, tokens, ids, cache, slots, table, lengths, q_start=None, last=None) -> Step:
        """fp32 logits behind tokens [n] (rows of several requests, one after the other);
        ids: their adapters; last: the rows that an answer is wanted for."""
        x = self.embed[tokens]
        c, s, g = self.qkv
        qkv = wush.linear_w4_lora(self.fmt, x, c, s, self.adapters, ids, T=self.qkv_T, global_scale=g)
        qkv = qkv.view(-1, self.q_heads + 2 * self.heads, self.D)
        q, k, v = qkv.split([self.q_heads, self.heads, self.heads], dim=1)
        wush.kv4_append(self.fmt, k, v, cache, slots, T_k=self.cache_T, T_v=self.cache_T)
        a = wush.kv4_attention(self.fmt, q, cache, table, lengths, q_start=q_start, T_q=self.cache_T)
        rows = a if last is None else a[last]
        x = x if last is None else x[last]
        c, s, g = self.out
        h = x + wush.linear_w4(self.fmt, rows.reshape(len(rows), -1), c, s, global_scale=g)
        c, s, g = self.head
        return Step(x, qkv, a, h, wush.linear_w4(self.fmt, h, c, s, global_scale=g, out_dtype=torch.float32))


def decode(block: Block, prompts, ids, steps: int, page: int = 64, penalty: float = 1.3, top: int = 5, look=None):
    """Greedy continuations of prompts (a list of int64 tensors), each with its adapter in
    ids (int32): (tokens [steps, requests], their log probabilities).  look, if given, is
    called with every step's parts."""
    dev, R = torch.device("cuda"), len(prompts)
    lengths = torch.tensor([len(p) for p in prompts], device=dev)
    width = (int(lengths.max()) + steps + page - 1) // page
    cache = block.cache(R * width, page)
    table = torch.arange(R * width, dtype=torch.int32, device=dev).view(R, width)
    start = torch.zeros(R + 1, dtype=torch.int32, device=dev)
    start[1:] = lengths.cumsum(0)
    request = torch.repeat_interleave(torch.arange(R, device=dev), lengths)
    place = torch.arange(len(request), device=dev) - start[request]
    asked = torch.full((R, int(lengths.max())), -1, dtype=torch.int32, device=dev)
    asked[request, place] = torch.cat(prompts).to(torch.int32)
    said = torch.full((R, steps), -1, dtype=torch.int32, device=dev)
    repetition, presence = torch.full((R,), penalty, device=dev), torch.full((R,), 0.1, device=dev)
    nothing = torch.full((R,), -1, device=dev)

    def slots(request, place):
        return table[request, place // page].long() * page + place % page

    call = dict(tokens=torch.cat(prompts), ids=ids[request], slots=slots(request, place), q_start=start, last=start[1:].long() - 1)
    tokens, logprobs = [], []
    everyone = torch.arange(R, device=dev)
    for n in range(steps):
        step = block.step(cache=cache, table=table, lengths=lengths.to(torch.int32), **call)
        logits = wush.adjust_logits(step.logits, prompt=asked, output=said, repetition=repetition, presence=presence)
        answer = wush.token_logprobs(logits, nothing, top=top)
        chosen = answer.top_ids[:, 0]
        if look is not None:
            look(n, call, step, cache, table, lengths, asked, said.clone(), logits, answer)
        tokens.append(chosen)
        logprobs.append(answer.top_logprobs[:, 0])
        said[:, n] = chosen
        call = dict(tokens=chosen.long(), ids=ids, slots=slots(everyone, lengths))
        lengths = lengths + 1
    return torch.stack(tokens), torch.stack(logprobs)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--fmt", choices=sorted(GROUP), default="mxfp4")
    p.add_argument("--vocab", type=int, default=32768)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--q-heads", type=int, default=32)
    p.add_argument("--heads", type=int, default=8)
    p.add_argument("--width", type=int, default=128)
    p.add_argument("--adapters", type=int, default=8)
    p.add_argument("--rank", type=int, default=16)
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--prompt", type=int, default=500)
    p.add_argument("--steps", type=int, default=16)
    a = p.parse_args(argv)
    block = Block(a.fmt, a.vocab, a.hidden, a.q_heads, a.heads, a.width, a.adapters, a.rank)
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompts = [torch.randint(0, a.vocab, (max(1, a.prompt * (r + 1) // a.requests),), generator=gen, device="cuda")
               for r in range(a.requests)]
    ids = torch.arange(a.requests, dtype=torch.int32, device="cuda") % (a.adapters + 1) - 1
    decode(block, prompts, ids, 2)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    tokens, logprobs = decode(block, prompts, ids, a.steps)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) * 1e3 / a.steps
    print("%s, %d requests of up to %d tokens: %.3f ms a step, the prompts among them; mean log probability %.4f"
          % (a.fmt, a.requests, a.prompt, ms, logprobs.mean()))
    return tokens, logprobs


if __name__ == "__main__":
    main()

"""The attention block of a decoder layer, served in 8 bits: block-scaled FP8
projections, a paged 8-bit key/value cache and attention that reads it.

A ragged batch of prompts is taken in one pass; then every sequence gets one new
token at a time, the step captured once as a graph and replayed.

    python examples/attention_block.py [--tokens 32] [--hidden 4096 --heads 32 --kv-heads 8]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w8a8_quantized_linear_channel_amd import ops as q8  # noqa: E402

PAGE = 64


class AttentionBlock:
    """x -> W_o attention(rotated W_q x, cached W_k x, cached W_v x)."""

    def __init__(self, w_qkv: torch.Tensor, w_out: torch.Tensor, heads: int, kv_heads: int, positions: int):
        self.heads, self.kv_heads, self.dim = heads, kv_heads, w_out.shape[1] // heads
        self.qkv, self.out = q8.q8_quantize_weight_block(w_qkv), q8.q8_quantize_weight_block(w_out)
        f = 10000.0 ** (-torch.arange(0, self.dim, 2, device=w_out.device, dtype=torch.float64) / self.dim)
        angle = torch.arange(positions, device=w_out.device, dtype=torch.float64)[:, None] * f
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def __call__(self, x: torch.Tensor, cache: q8.KvCache, batch: q8.KvBatch) -> torch.Tensor:
        h, hk = self.heads, self.kv_heads
        qkv = q8.q8_linear_fp8_block(x, *self.qkv).view(-1, h + 2 * hk, self.dim)
        q = q8.q8_kv_append(qkv[:, h:h + hk], qkv[:, h + hk:], cache, batch, q=qkv[:, :h], cos=self.cos, sin=self.sin)
        return q8.q8_linear_fp8_block(q8.q8_attention_kv8(q, cache, batch).flatten(1), *self.out)


class Sequences:
    """Pages and lengths of a batch that grows to at most `most` tokens a sequence."""

    def __init__(self, prompts, most: int, kv_heads: int, dim: int, device):
        n, pages = len(prompts), -(-most // PAGE)
        self.prompts, self.most = prompts, most
        self.cache = q8.q8_kv_cache(n * pages, kv_heads, dim, PAGE, device)
        self.table = torch.randperm(n * pages, device=device).int().view(n, pages)
        self.length = torch.zeros(n, dtype=torch.int32, device=device)
        self.one_each = torch.arange(n + 1, dtype=torch.int32, device=device)

    def prompt(self) -> q8.KvBatch:
        start = torch.zeros(len(self.prompts) + 1, dtype=torch.int32)
        start[1:] = torch.tensor(self.prompts).cumsum(0)
        self.length.copy_(torch.tensor(self.prompts, dtype=torch.int32))
        return q8.KvBatch(start.to(self.length.device), self.length, self.table, max(self.prompts), max(self.prompts))

    def next_token(self) -> q8.KvBatch:
        """One new token a sequence (the lengths are a tensor on the device, so a graph can hold this)."""
        self.length += 1
        return q8.KvBatch(self.one_each, self.length, self.table, 1, self.most)


def plain(x, w_qkv, w_out, heads, kv_heads, cos, sin):
    """One sequence [T, hidden] in binary32 without any quantization."""
    t, dim = x.shape[0], w_out.shape[1] // heads
    q, k, v = (x @ w_qkv.t()).view(t, -1, dim).split([heads, kv_heads, kv_heads], 1)

    def rotated(z):
        a, b = z.chunk(2, -1)
        c, s = cos[:t, None], sin[:t, None]
        return torch.cat((a * c - b * s, b * c + a * s), -1)
    q, k = rotated(q).transpose(0, 1), rotated(k).transpose(0, 1).repeat_interleave(heads // kv_heads, 0)
    s = (q @ k.transpose(1, 2).contiguous()) * dim ** -0.5
    s = s.masked_fill(torch.ones(t, t, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
    o = s.softmax(-1) @ v.transpose(0, 1).repeat_interleave(heads // kv_heads, 0)
    return o.transpose(0, 1).reshape(t, -1) @ w_out.t()


def run(hidden: int, heads: int, kv_heads: int, dim: int, prompts, tokens: int, device="cuda"):
    """(relative error against plain() over prompts and tokens, whether a replayed step gave the bits
    of an eager one, us of the prompt pass, us of a replayed step)"""
    gen = torch.Generator(device=device).manual_seed(0)
    w_qkv = torch.randn((heads + 2 * kv_heads) * dim, hidden, generator=gen, device=device) * hidden ** -0.5
    w_out = torch.randn(hidden, heads * dim, generator=gen, device=device) * (heads * dim) ** -0.5
    most = max(prompts) + tokens
    block = AttentionBlock(w_qkv, w_out, heads, kv_heads, most)
    xs = [torch.randn(n + tokens, hidden, generator=gen, device=device).bfloat16() for n in prompts]
    seqs = Sequences(prompts, most, kv_heads, dim, device)

    first = torch.cat([x[:n] for x, n in zip(xs, prompts)])
    batch = seqs.prompt()
    block(first, seqs.cache, batch)                  # writes the same tokens as the timed pass
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    y = block(first, seqs.cache, batch)
    torch.cuda.synchronize()
    prompt_us = (time.perf_counter() - t0) * 1e6

    step_x = torch.empty(len(prompts), hidden, dtype=torch.bfloat16, device=device)
    after_prompt = [c.clone() for c in seqs.cache]

    def back():
        for c, saved in zip(seqs.cache, after_prompt):
            c.copy_(saved)
        seqs.length.copy_(torch.tensor(prompts, dtype=torch.int32))

    def feed(i):
        step_x.copy_(torch.stack([x[n + i] for x, n in zip(xs, prompts)]))

    feed(0)
    eager = block(step_x, seqs.cache, seqs.next_token()).clone()
    back()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_y = block(step_x, seqs.cache, seqs.next_token())
    outs, step_us = [], 0.0
    for i in range(tokens):
        feed(i)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        graph.replay()
        torch.cuda.synchronize()
        step_us += (time.perf_counter() - t0) * 1e6 / tokens
        outs.append(step_y.clone())

    off = size = 0.0
    at = 0
    for s, n in enumerate(prompts):
        ref = plain(xs[s].float(), w_qkv, w_out, heads, kv_heads, block.cos, block.sin)
        got = torch.cat([y[at:at + n]] + [o[s:s + 1] for o in outs]).float()
        off, size, at = off + float((got - ref).square().sum()), size + float(ref.square().sum()), at + n
    return (off / size) ** 0.5, torch.equal(outs[0], eager), prompt_us, step_us


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--dim", type=int, default=128)
    p.add_argument("--prompts", type=int, nargs="+", default=[700, 33, 1, 512, 257, 1000, 64, 5])
    p.add_argument("--tokens", type=int, default=32)
    a = p.parse_args()
    err, same, prompt_us, step_us = run(a.hidden, a.heads, a.kv_heads, a.dim, a.prompts, a.tokens)
    print(f"{sum(a.prompts)} prompt tokens of {len(a.prompts)} sequences: {prompt_us:.0f} us; a step of one token each: "
          f"{step_us:.0f} us (replayed; eager bits {'the same' if same else 'DIFFER'}); "
          f"relative error against binary32: {err:.4f}")


if __name__ == "__main__":
    main()

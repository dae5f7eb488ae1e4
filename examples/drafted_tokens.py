"""Drafted tokens checked several at a time, and prompts that are sampled more than once, on a paged
8-bit cache: decoder layers' attention with normalised queries and keys.

The prompts are taken in one pass.  Then each is forked into samples that share its full pages.  A step
takes pages for a tree of drafts a sequence, appends them at their depth, lets each see the ones that it
continues, and moves those that are kept to the front.  It is captured once as a graph and replayed.

    python examples/drafted_tokens.py [--steps 16] [--samples 2] [--hidden 4096 --heads 32 --kv-heads 8]
"""
from __future__ import annotations

import argparse
import os
import random
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from w8a8_quantized_linear_channel_amd import ops as q8  # noqa: E402

PAGE = 32
EPS = 1e-6
# what each draft continues: the last token that is sure, two that may follow it, and so on
TREE = (-1, 0, 0, 0, 1, 1, 2, 4, 4, 7, 9)


def ancestors(tree):
    """(the drafts that each one sees as bits, its depth, the path that leads to it)"""
    paths = []
    for i, up in enumerate(tree):
        paths.append((paths[up] if up >= 0 else []) + [i])
    return [sum(1 << j for j in p) for p in paths], [len(p) - 1 for p in paths], paths


class NormedBlock:
    """x -> W_o attention(rotated norm(W_q x), cached rotated norm(W_k x), cached W_v x)."""

    def __init__(self, w_qkv, w_out, q_norm, k_norm, heads: int, kv_heads: int, angles):
        self.heads, self.kv_heads, self.dim = heads, kv_heads, w_out.shape[1] // heads
        self.qkv, self.out = q8.q8_quantize_weight_block(w_qkv), q8.q8_quantize_weight_block(w_out)
        self.q_norm, self.k_norm, (self.cos, self.sin) = q_norm, k_norm, angles

    def __call__(self, x, cache: q8.KvCache, batch: q8.KvBatch, positions=None, mask=None):
        h, hk = self.heads, self.kv_heads
        qkv = q8.q8_linear_fp8_block(x, *self.qkv).view(-1, h + 2 * hk, self.dim)
        q = q8.q8_kv_append_norm(qkv[:, h:h + hk], qkv[:, h + hk:], cache, batch, q=qkv[:, :h], q_weight=self.q_norm,
                                 k_weight=self.k_norm, eps=EPS, cos=self.cos, sin=self.sin, positions=positions)
        y = (q8.q8_attention_kv8(q, cache, batch) if mask is None else
             q8.q8_attention_kv8_tree(q, cache, batch, mask, positions=positions))
        return q8.q8_linear_fp8_block(y.flatten(1), *self.out)


def plain(x, w_qkv, w_out, q_norm, k_norm, heads, kv_heads, cos, sin):
    """One sequence [T, hidden] in binary32 without any quantization."""
    t, dim = x.shape[0], w_out.shape[1] // heads
    q, k, v = (x @ w_qkv.t()).view(t, -1, dim).split([heads, kv_heads, kv_heads], 1)

    def turned(z, w):
        z = z * (z.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
        a, b = z.chunk(2, -1)
        c, s = cos[:t, None], sin[:t, None]
        return torch.cat((a * c - b * s, b * c + a * s), -1)
    q, k = turned(q, q_norm).transpose(0, 1), turned(k, k_norm).transpose(0, 1).repeat_interleave(heads // kv_heads, 0)
    s = (q @ k.transpose(1, 2).contiguous()) * dim ** -0.5
    s = s.masked_fill(torch.ones(t, t, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
    o = s.softmax(-1) @ v.transpose(0, 1).repeat_interleave(heads // kv_heads, 0)
    return o.transpose(0, 1).reshape(t, -1) @ w_out.t()


class Drafts:
    """The samples' batch between steps, in tensors that a graph can hold, and one step of it."""

    def __init__(self, layers, caches, sequences: q8.KvFork, hidden: int):
        dev = sequences.kv_len.device
        self.layers, self.caches, self.n = layers, caches, len(TREE)
        self.table, self.length, self.refs, self.missing = (t.clone() for t in sequences)
        self.seqs, self.most = self.table.shape[0], self.table.shape[1] * PAGE
        bits, depth, self.paths = ancestors(TREE)
        self.mask = torch.tensor(bits, device=dev)[None].repeat(self.seqs, 1).view(-1, 1)
        self.depth = torch.tensor(depth, dtype=torch.int32, device=dev)
        self.parent = torch.arange(self.seqs, dtype=torch.int32, device=dev)
        self.start = torch.arange(self.seqs + 1, dtype=torch.int32, device=dev) * self.n
        self.x = torch.zeros(self.seqs * self.n, hidden, dtype=torch.bfloat16, device=dev)
        self.keep = torch.zeros(self.seqs, max(depth) + 1, dtype=torch.int32, device=dev)
        self.kept = torch.ones(self.seqs, dtype=torch.int32, device=dev)

    def feed(self, x, chosen):
        """The drafts' inputs, and the draft each sequence ends with."""
        self.x.copy_(x)
        width = self.keep.shape[1]
        self.keep.copy_(torch.tensor([self.paths[c] + [-1] * (width - len(self.paths[c])) for c in chosen]))
        self.kept.copy_(torch.tensor([len(self.paths[c]) for c in chosen]))

    def step(self):
        """[(input, output) of each layer]"""
        new = q8.q8_kv_fork(self.caches, self.table, self.length, self.refs, self.parent, room=self.n)
        batch = q8.KvBatch(self.start, new.kv_len + self.n, new.block_table, self.n, self.most)
        positions = (new.kv_len[:, None] + self.depth).flatten()
        x, seen = self.x, []
        for layer, cache in zip(self.layers, self.caches):
            y = layer(x, cache, batch, positions, self.mask)
            seen.append((x, y))
            x = x + y
        q8.q8_kv_compact(self.caches, batch, self.keep, self.kept, out=self.length)
        self.table.copy_(new.block_table)
        self.refs.copy_(new.refs)
        self.missing.add_(new.missing)
        return seen

    def state(self):
        return [self.table, self.length, self.refs, self.missing] + [t for c in self.caches for t in c]


def run(hidden: int, heads: int, kv_heads: int, dim: int, prompts, samples: int, steps: int, layers: int = 2, device="cuda"):
    """(the layers' relative error against plain() on the inputs that they had, over prompts and kept
    tokens; whether a replayed step gave the bits of an eager one; whether the tables were right at the end;
    tokens kept a step and sequence; us of a replayed step)"""
    gen = torch.Generator(device=device).manual_seed(0)
    pick = random.Random(0)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=device)

    bits, depth, paths = ancestors(TREE)
    n, S = len(TREE), len(prompts) * samples
    most = max(prompts) + (max(depth) + 1) * steps + n
    width = -(-most // PAGE)
    pages = len(prompts) * width * samples
    f = 10000.0 ** (-torch.arange(0, dim, 2, device=device, dtype=torch.float64) / dim)
    angle = torch.arange(most, device=device, dtype=torch.float64)[:, None] * f
    angles = angle.cos().float(), angle.sin().float()
    weights = [(normal((heads + 2 * kv_heads) * dim, hidden) * hidden ** -0.5, normal(hidden, heads * dim) * (heads * dim) ** -0.5,
                1 + normal(dim) / 8, 1 + normal(dim) / 8) for _ in range(layers)]
    blocks = [NormedBlock(*w, heads, kv_heads, angles) for w in weights]
    caches = [q8.q8_kv_cache(pages, kv_heads, dim, PAGE, device) for _ in range(layers)]

    def ints(a):
        return torch.tensor(a, dtype=torch.int32, device=device)

    # pages for the prompts: a batch without a token and without a page, continued with room for them
    nothing = q8.KvFork(torch.full((len(prompts), width), -1, dtype=torch.int32, device=device), ints([0] * len(prompts)),
                        ints([0] * pages), ints([0]))
    batch = q8.q8_kv_fork(caches, *nothing[:3], ints(range(len(prompts))), room=max(prompts))
    lens, ends = ints(prompts), ints([0] + prompts).cumsum(0).int()
    x = normal(sum(prompts), hidden).bfloat16()
    history = [[[] for _ in range(layers)] for _ in prompts]            # [sequence][layer]: (input, output)
    for i, (block, cache) in enumerate(zip(blocks, caches)):
        y = block(x, cache, q8.KvBatch(ends, lens, batch.block_table, max(prompts), max(prompts)))
        for s, (a, b) in enumerate(zip(x.split(prompts), y.split(prompts))):
            history[s][i].append((a, b))
        x = x + y

    # each prompt goes on as `samples` sequences
    parents = [s for s in range(len(prompts)) for _ in range(samples)]
    forked = q8.q8_kv_fork(caches, batch.block_table, lens, batch.refs, ints(parents))
    history = [[list(h) for h in history[p]] for p in parents]
    drafts = Drafts(blocks, caches, forked, hidden)

    def inputs():
        return normal(S * n, hidden).bfloat16(), [pick.randrange(n) for _ in range(S)]

    given = inputs()
    drafts.feed(*given)
    before = [t.clone() for t in drafts.state()]

    def back():
        for t, saved in zip(drafts.state(), before):
            t.copy_(saved)

    eager = [t.clone() for xy in drafts.step() for t in xy] + [t.clone() for t in drafts.state()]
    back()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        seen = drafts.step()
    same, step_us, kept = True, 0.0, 0
    for i in range(steps):
        if i > 0:
            given = inputs()
            drafts.feed(*given)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        graph.replay()
        torch.cuda.synchronize()
        step_us += (time.perf_counter() - t0) * 1e6 / steps
        if i == 0:
            replayed = [t for xy in seen for t in xy] + drafts.state()
            same = all(torch.equal(a, b) for a, b in zip(eager, replayed))
        for s, end in enumerate(given[1]):
            rows = torch.tensor(paths[end], device=device) + s * n
            kept += len(paths[end])
            for layer, (a, b) in zip(history[s], seen):
                layer.append((a[rows], b[rows]))

    # the tables: no page is missing, each is counted as often as it is held, only full pages of a prompt are shared
    held = drafts.table[drafts.table >= 0].long()
    right = int(drafts.missing) == 0 and torch.equal(torch.bincount(held, minlength=pages).int(), drafts.refs)
    right &= drafts.length.tolist() == [sum(a.shape[0] for a, _ in h[0]) for h in history]
    right &= int((drafts.refs > 1).sum()) == (sum(p // PAGE for p in prompts) if samples > 1 else 0)
    off = size = 0.0
    for h in history:
        for w, layer in zip(weights, h):
            a, b = (torch.cat(t).float() for t in zip(*layer))
            ref = plain(a, *w, heads, kv_heads, *angles)
            off, size = off + float((b - ref).square().sum()), size + float(ref.square().sum())
    return (off / size) ** 0.5, same, bool(right), kept / (steps * S), step_us


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--dim", type=int, default=128)
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--prompts", type=int, nargs="+", default=[700, 33, 1, 512])
    p.add_argument("--samples", type=int, default=2)
    p.add_argument("--steps", type=int, default=16)
    a = p.parse_args()
    err, same, right, kept, step_us = run(a.hidden, a.heads, a.kv_heads, a.dim, a.prompts, a.samples, a.steps, a.layers)
    print(f"{len(a.prompts)} prompts sampled {a.samples} times, {a.layers} layers: a step of {len(TREE)} drafts a sequence "
          f"{step_us:.0f} us (replayed; eager bits {'the same' if same else 'DIFFER'}), {kept:.2f} tokens kept of it; "
          f"tables {'right' if right else 'WRONG'}; relative error against binary32: {err:.4f}")


if __name__ == "__main__":
    main()

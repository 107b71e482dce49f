"""The attention of a decode step over a paged cache in MXFP4, from the layer's input to its output.

    project   mx_quantize_rows, mx_gemm: query latent and key/value latent of each token
    queries   mx_rmsnorm_quantize_rows, mx_gemm: 16 heads of 512 dimensions
    rotate    mx_rope: the last 64 dimensions of the query heads and of the latent
    write     mx_cache_write: the latent into its slot, 272 bytes
    attend    mx_attend: all heads over the one latent of each cached token
    output    wo_a_grouped (which undoes the rotation of what was summed), mx_gemm

A latent is key and value in one. Prompts and single tokens take the same calls: a step is any
number of tokens of any sequences. With fixed buffers it also runs as a CUDA graph, in which the
sequences grow from replay to replay.

    python examples/cached_attention.py --sequences 4 --prompt 100 --steps 20
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import mxfp8_block_scaled_06_gb300 as mx

HEADS, D, D_ROPE, LATENT = 16, 512, 64, 1536  # query heads and their dimensions, rotated ones, query latent
MOST_ROWS = 256  # of one projection's call


class CachedAttention:
    """One layer's attention with its cache. hidden % 128 == 0; rank: of the grouped output projection."""

    def __init__(self, handle, hidden, rank=256, pages=64, page_size=64, max_pos=4096, seed=0):
        self.h, self.rank = handle, rank
        g = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda n, k: mx.mx_quantize_rows(handle, (torch.randn(n, k, generator=g, device="cuda")  # noqa: E731
                                                         * k ** -0.5).bfloat16())
        self.wa, self.wq = make(LATENT + D, hidden), make(HEADS * D, LATENT)
        self.wo_a, self.wo_b = make(2 * rank, HEADS // 2 * D), make(hidden, 2 * rank)
        self.norm = torch.ones(LATENT, dtype=torch.bfloat16, device="cuda")
        self.cos_sin = mx.mx_rope_table(handle, max_pos, D_ROPE, scaling="yarn", factor=4.0, original=max_pos // 4)
        self.cache = mx.MxCache.zeros(handle, pages, page_size, 1, D, shared=True)

    def _project(self, rows, weight):
        return torch.cat([mx.mx_gemm(self.h, *mx.mx_quantize_rows(self.h, part), *weight) for part in rows.split(MOST_ROWS)])

    def __call__(self, x, positions, slots, table, lengths, q_offsets=None, parts=None):
        """x [T, hidden] bf16; each token's position and slot; each sequence's pages and cached tokens, these among
        them. A dict given as parts gets what the steps hand on."""
        h, t = self.h, x.shape[0]
        a = self._project(x, self.wa)
        q = torch.cat([mx.mx_gemm(h, *mx.mx_rmsnorm_quantize_rows(h, part, self.norm, 1e-6)[:2], *self.wq)
                       for part in a[:, :LATENT].split(MOST_ROWS)]).view(t, HEADS, D)
        latent = a[:, LATENT:].view(t, 1, D)
        q = mx.mx_rope(h, q, positions, self.cos_sin, out=q)
        latent = mx.mx_rope(h, latent, positions, self.cos_sin)
        mx.mx_cache_write(h, self.cache, slots, latent)
        out = mx.mx_attend(h, q, self.cache, table, lengths, q_offsets=q_offsets)
        ys = []
        for i in range(0, t, MOST_ROWS):
            part = slice(i, i + MOST_ROWS)
            z = mx.wo_a_grouped_unfused(h, out[part], positions[part], self.cos_sin, *self.wo_a, 2, HEADS // 2, self.rank)
            ys.append(mx.mx_gemm(h, z["q"], z["q_scales"], *self.wo_b))
        if parts is not None:
            parts.update(q=q, latent=latent, out=out)
        return torch.cat(ys)


def place(table, page_size, seq, pos):
    """Slots of tokens at positions pos of sequences seq."""
    return table[seq, pos // page_size].long() * page_size + pos % page_size


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--hidden", type=int, default=1024)
    a = ap.parse_args()
    torch.cuda.set_device(0)
    h = mx.mx_create(0)
    b, page = a.sequences, 64
    columns = (a.prompt + a.steps + 1 + page - 1) // page
    layer = CachedAttention(h, a.hidden, pages=b * columns, page_size=page, max_pos=columns * page)
    table = torch.randperm(b * columns, device="cuda").int().view(b, columns)
    # prompts of different lengths in one step
    counts = [max(1, a.prompt - 7 * i) for i in range(b)]
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), torch.tensor(counts, device="cuda"))
    pos = torch.cat([torch.arange(n, device="cuda") for n in counts])
    lengths = torch.tensor(counts, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([sum(counts[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
    layer(torch.randn(len(pos), a.hidden, device="cuda").bfloat16(), pos, place(table, page, seq, pos), table, lengths, offsets)

    # single tokens: one graph, whose sequences are a token longer with each replay
    x, every = torch.randn(b, a.hidden, device="cuda").bfloat16(), torch.arange(b, device="cuda")

    def step():
        where = lengths.long()
        lengths.add_(1)
        return layer(x, where, place(table, page, every, where), table, lengths)

    before = lengths.clone()
    eager = step().clone()
    lengths.copy_(before)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    lengths.copy_(before)
    graph.replay()
    torch.cuda.synchronize()
    same = torch.equal(out, eager)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if mx.mx_device_status(h) != mx.MX_OK or not same or not torch.isfinite(out).all():
        raise SystemExit("the graph's result differs from the eager one")
    print(f"{b} sequences of {counts[0]} tokens and fewer: {begin.elapsed_time(end) * 1e3 / a.steps:.1f} us a step")


if __name__ == "__main__":
    main()

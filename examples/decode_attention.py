"""Decode with a paged K/V cache: the attention block of a decoder layer for a batch of sequences.

    python examples/decode_attention.py [--seqs 32] [--prompt 1000] [--steps 50] [--cache q8]

Each step is six calls on one stream, captured once as a CUDA graph and replayed:

    q, k, v = x Wq^T, x Wk^T, x Wv^T    one shared-input batch (matmul_batch)
    kv_extend                           every sequence one token longer: pages, block table, slots
    kv_append                           k and v into the slots
    kv_attend                           q over each sequence's cache
    o = attention Wo^T                  the next batch

The lengths and the block table live on the GPU; the host does nothing between steps but
replay.  Positions are not encoded (a model rotates q and k before the last three calls).
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import shared_input_linear_gb300 as sil  # noqa: E402


class AttentionBlock:
    """q/k/v and output projections of one layer, and the cache of up to ``n_seq`` sequences."""

    def __init__(self, n_in=4096, heads=32, kv_heads=8, dim=128, n_seq=32, page=16, pages=4096, cache="q8", seed=0):
        self.n_in, self.heads, self.kv_heads, self.dim, self.n_seq, self.page = n_in, heads, kv_heads, dim, n_seq, page
        gen = torch.Generator().manual_seed(seed)

        def weight(n_out, width):  # N(0, 1 / width) rounded to bf16, as the host has it
            w = (torch.randn((n_out, width), generator=gen) * width ** -0.5).bfloat16()
            return w, sil.upload_weight("bf16", w.view(torch.int16).numpy().view(np.uint16), n_out, width)

        self.host, self.dev = zip(*(weight(n, n_in) for n in (heads * dim, kv_heads * dim, kv_heads * dim)))
        self.host_o, self.w_o = weight(n_in, heads * dim)
        self.cache = sil.kv_cache(cache, pages, page, kv_heads, dim)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(n_seq, **i32)
        self.table = torch.zeros((n_seq, pages // n_seq), **i32)
        self.ring = torch.arange(pages, **i32)
        self.cursor = torch.tensor([0, pages], dtype=torch.int64, device="cuda")
        self.info = torch.zeros(4, dtype=torch.int64, device="cuda")
        self.one = torch.ones(n_seq, **i32)
        self.slots = torch.empty(n_seq, **i32)
        f32 = dict(device="cuda")
        self.x = torch.zeros((n_seq, n_in), **f32)
        self.q, self.k, self.v = (torch.empty((n_seq, h * dim), **f32) for h in (heads, kv_heads, kv_heads))
        self.attention = torch.empty((n_seq, heads, dim), **f32)
        self.out = torch.empty((n_seq, n_in), **f32)

    def prompt(self, x, lens):
        """The prompts' tokens, one sequence after the other ``[sum(lens)][n_in]``, into the cache."""
        n = x.shape[0]
        k, v = (torch.empty((n, self.kv_heads * self.dim), device="cuda") for _ in range(2))
        sil.matmul_batch(x, [(self.dev[1], k), (self.dev[2], v)])
        slots = torch.empty(n, dtype=torch.int32, device="cuda")
        add = torch.tensor(lens, dtype=torch.int32, device="cuda")
        sil.kv_extend(self.lens, add, self.table, self.ring, self.cursor, self.page, slots, info=self.info)
        if int(self.info[0]) != 0:
            raise RuntimeError(f"the cache has no room for the prompts: {self.info.tolist()}")
        sil.kv_append(self.cache, k, v, slots)

    def step(self):
        """One token of every sequence: reads ``x``, writes ``out``."""
        sil.matmul_batch(self.x, list(zip(self.dev, (self.q, self.k, self.v))))
        sil.kv_extend(self.lens, self.one, self.table, self.ring, self.cursor, self.page, self.slots, info=self.info)
        sil.kv_append(self.cache, self.k, self.v, self.slots)
        sil.kv_attend(self.cache, self.q.view(self.n_seq, self.heads, self.dim), self.table, self.lens, self.attention)
        sil.matmul_batch(self.attention.view(self.n_seq, -1), [(self.w_o, self.out)])

    def finish(self, which):
        """Sequences ``which`` give their pages back."""
        add = torch.zeros(self.n_seq, dtype=torch.int32, device="cuda")
        add[list(which)] = -2**31
        sil.kv_extend(self.lens, add, self.table, self.ring, self.cursor, self.page, self.slots, info=self.info)

    def capture(self):
        """A graph of :meth:`step`.  One step runs first, so that the library's workspaces exist, and is taken back."""
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())  # for the prompts' last kv_append, and x
        with torch.cuda.stream(stream):
            self.step()
            sil.kv_extend(self.lens, -self.one, self.table, self.ring, self.cursor, self.page, self.slots)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                self.step()
        return graph


def main(argv=None) -> dict:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=1000, help="longest prompt")
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--cache", choices=("bf16", "q8"), default="q8")
    a = ap.parse_args(argv)
    page = 16
    pages = a.seqs * (-(-(a.prompt + a.steps + 2) // page) + 1)
    block = AttentionBlock(n_seq=a.seqs, page=page, pages=pages, cache=a.cache)
    gen = torch.Generator(device="cuda").manual_seed(1)
    lens = [a.prompt - (i * a.prompt) // (2 * a.seqs) for i in range(a.seqs)]
    for i in range(a.seqs):  # one prompt at a time, as they arrive
        add = [0] * a.seqs
        add[i] = lens[i]
        block.prompt(torch.randn((lens[i], block.n_in), generator=gen, device="cuda"), add)
    graph = block.capture()
    block.x.copy_(torch.randn(block.x.shape, generator=gen, device="cuda"))
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    sil.check_device_status()
    if block.lens.tolist() != [n + a.steps for n in lens] or int(block.info[0]) != 0:
        raise RuntimeError("a step had no room in the cache")
    us = begin.elapsed_time(end) * 1e3 / a.steps
    print(f"{a.seqs} sequences of {min(lens)} to {max(lens)} tokens, {a.cache} cache: {us:.1f} us a step, "
          f"{a.seqs / us * 1e6:.0f} tokens/s through one layer's attention block")
    return {"us": us, "block": block}


if __name__ == "__main__":
    main()

#!/usr/bin/env python3
"""One layer's attention block on int4 weights, for prompts and for single tokens.

    x -> fused q/k/v/gate/up product -> head norm, rotary position, cache append
      -> attention over the paged cache -> o_proj

with the shapes of the rumik-oss-1 write-up's model (hidden size 2,048; the fused
25,088-row matrix holds 16 query and 4 key and value heads of 128, then the gate
and up rows, which this block leaves alone).  Two requests are prompted in one
call and then decoded together, one token each per step; a token's next input
stands in for the rest of the model (its own normalised output).  At the end the
same tokens go through the prompt path in one piece, which has to give the same
outputs.

    python examples/attention_block.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

import int4_group_quantized_amd as q4  # noqa: E402
import synth  # noqa: E402

HEADS, KV_HEADS, DIM, PAGE = 16, 4, 128, 64


def rope_frequencies(dim: int, base: float = 10000.0, factor: float = 1.0) -> torch.Tensor:
    """Inverse frequencies [dim / 2]; factor > 1 stretches all positions for a longer context."""
    return (base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim) / factor).float()


class Matrix:
    """An int4 matrix on the GPU."""

    def __init__(self, w, dev):
        self.packed = q4.q4g128_pack(torch.from_numpy(w.codes).to(dev))
        self.scales, self.mins = torch.from_numpy(w.scales).to(dev), torch.from_numpy(w.mins).to(dev)

    def __call__(self, x):
        """x fp16 [T][K] -> fp32 [T][N]: the small-batch product up to 16 rows, else the prompt product."""
        product = q4.q4g128_gemm_small_batch if x.shape[0] <= q4.MAX_BATCH else q4.q4g128_gemm_prefill_epilogue
        return product(self.packed, self.scales, self.mins, x)


class AttentionBlock:
    """Weights, page pool and page tables of up to `sequences` requests."""

    def __init__(self, dev, sequences=4, pages=32, max_length=1024):
        self.fused = Matrix(synth.weights(synth.FUSED_N, synth.PAGES_HIDDEN, synth.SEEDS["pages_fused"]), dev)
        self.o_proj = Matrix(synth.weights(synth.PAGES_HIDDEN, HEADS * DIM, synth.SEEDS["pages_oproj"]), dev)
        self.k = torch.empty((pages, KV_HEADS, PAGE, DIM), dtype=torch.float16, device=dev)
        self.v = torch.empty((pages, KV_HEADS, DIM, PAGE), dtype=torch.float16, device=dev)
        self.table = torch.full((sequences, max_length // PAGE), -1, dtype=torch.int32, device=dev)
        self.free = list(range(pages))
        self.held = [[] for _ in range(sequences)]
        self.length = [0] * sequences
        self.freq = rope_frequencies(DIM).to(dev)
        self.norm = torch.ones(DIM, dtype=torch.float16, device=dev)
        self.dev = dev

    def _grow(self, s, tokens):
        """Pages for `tokens` more positions of sequence s; returns the first new position."""
        first = self.length[s]
        self.length[s] += tokens
        while len(self.held[s]) * PAGE < self.length[s]:
            self.held[s].append(self.free.pop())
        self.table[s, :len(self.held[s])] = torch.tensor(self.held[s], dtype=torch.int32, device=self.dev)
        return first

    def release(self, s):
        """Sequence s ends: its pages go back."""
        self.free += self.held[s]
        self.held[s], self.length[s] = [], 0
        self.table[s] = -1

    def _ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.dev)

    def prompt(self, xs):
        """xs: fp16 [T_s][2048] of sequences 0, 1, ...; returns their outputs fp32 [T_s][2048]."""
        new = [len(x) for x in xs]
        firsts = [self._grow(s, n) for s, n in enumerate(new)]
        seq = self._ints([s for s, n in enumerate(new) for _ in range(n)])
        positions = self._ints([f + i for f, n in zip(firsts, new) for i in range(n)])
        starts = self._ints([sum(new[:s]) for s in range(len(new) + 1)])
        q = q4.q4g128_rope_append(self.fused(torch.cat(xs)), self.k, self.v, self.table, positions, self.freq, HEADS,
                                  seq=seq, q_norm=self.norm, k_norm=self.norm)
        lengths = self.length[:len(xs)]
        out = q4.q4g128_attn_prefill(q, self.k, self.v, self.table, starts, self._ints(lengths),
                                     max_length=max(lengths))
        return self.o_proj(out.view(sum(new), HEADS * DIM)).split(new)

    def step(self, x):
        """x fp16 [B][2048], one token of each of the sequences 0 .. B-1; returns fp32 [B][2048]."""
        b = x.shape[0]
        positions = self._ints([self._grow(s, 1) for s in range(b)])
        q = q4.q4g128_rope_append(self.fused(x), self.k, self.v, self.table, positions, self.freq, HEADS,
                                  q_norm=self.norm, k_norm=self.norm)
        out = q4.q4g128_attn_decode(q, self.k, self.v, self.table, positions + 1, max_length=max(self.length))
        return self.o_proj(out.view(b, HEADS * DIM))


def next_input(y):
    """Stand-in for the rest of the model: the normalised output, fp16."""
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True))).half()


def main(steps=8):
    """Returns the largest difference between the decoded outputs and the prompt path's, over their rms."""
    dev = torch.device("cuda")
    block = AttentionBlock(dev)
    prompts = [torch.from_numpy(synth.activations(n, synth.PAGES_HIDDEN, 90 + n)).to(dev) for n in (34, 21)]
    first = block.prompt(prompts)
    x = next_input(torch.stack([y[-1] for y in first]))
    inputs, outputs = [], []
    for _ in range(steps):
        inputs.append(x)
        outputs.append(block.step(x))
        x = next_input(outputs[-1])
    # The whole sequences again, in one prompt call on an empty cache.
    for s in range(len(prompts)):
        block.release(s)
    whole = block.prompt([torch.cat([p] + [i[s:s + 1] for i in inputs]) for s, p in enumerate(prompts)])
    worst = 0.0
    for s, p in enumerate(prompts):
        got = torch.cat([first[s]] + [o[s:s + 1] for o in outputs])
        want = whole[s]
        worst = max(worst, ((got - want).abs().max() / want.square().mean().sqrt()).item())
    torch.cuda.synchronize()
    return worst


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=8)
    print(f"decoded outputs within {main(parser.parse_args().steps):.2e} of the prompt path's (of their rms)")

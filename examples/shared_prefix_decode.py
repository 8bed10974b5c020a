"""Attention side of a decoder layer on 4-bit weights, for a batch that shares a prompt.

One layer of a decoder (12 query and 2 key/value heads of 128 elements, hidden size 1536): the
prompt's keys and values are appended to a paged cache once; then every step takes one token of
each sequence through the fused q/k/v GEMVs, ``nf4_kv_append`` (norm, rotation, append) ,
``nf4_prefix_attention`` and the o GEMV, recorded once into a CUDA graph and replayed.

    python examples/shared_prefix_decode.py [--batch 32] [--prompt 8192] [--steps 64]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import w4a16_gemv_gb300 as nf4  # noqa: E402

PAGE = 16


class AttentionLayer:
    """Weights, cache and page tables of one layer for `batch` sequences over one prompt."""

    def __init__(self, batch: int, prompt: int, most_new: int, hidden: int = 1536, q_heads: int = 12, kv_heads: int = 2,
                 dim: int = 128, seed: int = 1):
        dev = torch.device("cuda")
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        code2 = torch.tensor([(i - 127.5) / 127.5 for i in range(256)], dtype=torch.float16, device=dev)

        def weight(n, k):
            w = torch.randn(n, k, device=dev, generator=gen) / k ** 0.5
            return nf4.nf4_quantize(w, code2)
        self.q_heads, self.kv_heads, self.dim, self.batch, self.prompt = q_heads, kv_heads, dim, batch, prompt
        self.wq, self.wk = weight(q_heads * dim, hidden), weight(kv_heads * dim, hidden)
        self.wv, self.wo = weight(kv_heads * dim, hidden), weight(hidden, q_heads * dim)
        self.q_norm = (1 + 0.1 * torch.randn(dim, device=dev, generator=gen)).bfloat16()
        self.k_norm = (1 + 0.1 * torch.randn(dim, device=dev, generator=gen)).bfloat16()
        self.cos_sin = nf4.nf4_rope_table(prompt + most_new, dim, base=1e6)
        # pages: the prompt's first, then each sequence's own
        shared, own = -(-prompt // PAGE), -(-most_new // PAGE)
        self.prefix_pages = torch.arange(shared, dtype=torch.int32, device=dev)
        self.suffix_pages = shared + torch.arange(batch * own, dtype=torch.int32, device=dev).view(batch, own)
        self.k_cache = torch.empty(shared + batch * own, PAGE, kv_heads, dim, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.empty_like(self.k_cache)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)  # own keys of each sequence

    def gemv(self, weight, x, heads=None):
        """The fused GEMV in slabs of its widest batch."""
        y = torch.cat([nf4.gemv(weight, x[i:i + 64], out_dtype=torch.bfloat16) for i in range(0, x.shape[0], 64)])
        return y if heads is None else y.view(x.shape[0], heads, self.dim)

    def read_prompt(self, x: torch.Tensor) -> None:
        """Appends the prompt's keys and values (x: bf16 [prompt, hidden])."""
        at = torch.arange(self.prompt, device=x.device)
        nf4.nf4_kv_append(self.k_cache, self.v_cache, at, self.gemv(self.wk, x, self.kv_heads),
                          self.gemv(self.wv, x, self.kv_heads), at, self.cos_sin, k_weight=self.k_norm)

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """One token of each sequence: bf16 [batch, hidden] in and out. Lengths live on the device and grow there,
        so that a recorded step can be replayed."""
        n = self.lens.long()
        slots = self.suffix_pages.gather(1, (n // PAGE)[:, None])[:, 0].long() * PAGE + n % PAGE
        q = nf4.nf4_kv_append(self.k_cache, self.v_cache, slots, self.gemv(self.wk, x, self.kv_heads),
                              self.gemv(self.wv, x, self.kv_heads), self.prompt + n, self.cos_sin,
                              q=self.gemv(self.wq, x, self.q_heads), q_weight=self.q_norm, k_weight=self.k_norm)
        self.lens += 1
        out = nf4.nf4_prefix_attention(q, self.k_cache, self.v_cache, self.prefix_pages, self.prompt, self.suffix_pages,
                                       self.lens)
        return self.gemv(self.wo, out.view(self.batch, -1))


def run(batch: int, prompt: int, steps: int, seed: int = 1):
    """Reads a prompt and decodes `steps` tokens per sequence; returns (layer, prompt inputs, inputs and outputs of
    the steps, us per step)."""
    layer = AttentionLayer(batch, prompt, steps, seed=seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    hidden = layer.wq.shape[1]
    x_prompt = torch.randn(prompt, hidden, device="cuda", generator=gen).bfloat16()
    xs = torch.randn(steps, batch, hidden, device="cuda", generator=gen).bfloat16()
    layer.read_prompt(x_prompt)
    x, ys = xs[0].clone(), torch.empty_like(xs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x)  # once outside the recording: modules load, allocations settle
        layer.lens.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = layer.step(x)
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record(side)
        for i in range(steps):
            x.copy_(xs[i])
            graph.replay()
            ys[i].copy_(y)
        end.record(side)
    side.synchronize()
    if nf4.nf4_device_error_flags() != 0:
        raise RuntimeError("device error flags set")
    return layer, x_prompt, xs, ys, start.elapsed_time(end) * 1e3 / steps


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=64)
    args = ap.parse_args()
    _, _, _, ys, us = run(args.batch, args.prompt, args.steps)
    print(f"{args.batch} sequences over a shared prompt of {args.prompt}: {us:.1f} us per step and layer "
          f"(attention side), mean |y| {ys.float().abs().mean():.4f}")


if __name__ == "__main__":
    main()

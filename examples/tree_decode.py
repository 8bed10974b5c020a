"""Speculative decoding with drafted trees on 4-bit weights, for a batch over one prompt.

One layer of a decoder (12 query and 2 key/value heads of 128 elements, hidden size 1536) with its embedding and
its output head. Every step drafts a tree of tokens per sequence from a table of likely followers, lays the tree
out in the paged cache (``nf4_kv_pages``), takes all its nodes through the layer at once (the fused GEMVs,
``nf4_kv_append``, ``nf4_tree_attention``), penalises repeated tokens and picks each node's best next one
(``nf4_adjust_logits``), and keeps the branch that the model agrees with (``nf4_tree_commit``). A step reads
nothing back, so it is recorded once into a CUDA graph and replayed: each replay adds one to four tokens to every
sequence, and pages come and go as the sequences grow.

    python examples/tree_decode.py [--batch 16] [--prompt 1000] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import w4a16_gemv_gb300 as nf4  # noqa: E402

PAGE = 16
# A node's parent, and which of its parent's followers it holds: two levels of three, and one below.
TREE = [(0, 0), (0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (2, 0), (4, 0)]
LEVELS = [range(1, 4), range(4, 7), range(7, 8)]


class TreeDecoder:
    """Weights, cache and state of `batch` sequences over one prompt (token numbers, int64 [prompt])."""

    def __init__(self, batch: int, prompt: torch.Tensor, most_new: int, vocab: int = 2000, hidden: int = 1536,
                 q_heads: int = 12, kv_heads: int = 2, dim: int = 128, seed: int = 1):
        dev = torch.device("cuda")
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        code2 = torch.tensor([(i - 127.5) / 127.5 for i in range(256)], dtype=torch.float16, device=dev)

        def weight(n, k):
            return nf4.nf4_quantize(torch.randn(n, k, device=dev, generator=gen) / k ** 0.5, code2)

        def ints(v):
            return torch.tensor(v, dtype=torch.int32, device=dev)
        self.q_heads, self.kv_heads, self.dim, self.batch, self.prompt = q_heads, kv_heads, dim, batch, prompt.numel()
        self.wq, self.wk = weight(q_heads * dim, hidden), weight(kv_heads * dim, hidden)
        self.wv, self.wo = weight(kv_heads * dim, hidden), weight(hidden, q_heads * dim)
        self.head = weight(vocab, hidden)
        self.embed = torch.randn(vocab, hidden, device=dev, generator=gen).bfloat16()
        self.q_norm = (1 + 0.1 * torch.randn(dim, device=dev, generator=gen)).bfloat16()
        self.k_norm = (1 + 0.1 * torch.randn(dim, device=dev, generator=gen)).bfloat16()
        n = len(TREE)
        self.cos_sin = nf4.nf4_rope_table(self.prompt + most_new + n, dim, base=1e6)
        # what is likely to follow a token, from its embedding alone
        self.followers = self.gemv(self.head, self.embed, torch.float32).topk(3, 1).indices.int()
        # pages: the prompt's first; the others are free
        shared, width = -(-self.prompt // PAGE), -(-(most_new + n) // PAGE)
        pages = shared + batch * width
        self.prefix_pages = torch.arange(shared, dtype=torch.int32, device=dev)
        self.k_cache = torch.zeros(pages, PAGE, kv_heads, dim, dtype=torch.bfloat16, device=dev)
        self.v_cache = torch.zeros_like(self.k_cache)
        self.free_pages, self.free_count = torch.arange(shared, pages, dtype=torch.int32, device=dev), ints([pages - shared])
        self.page_table = torch.zeros(batch, width, dtype=torch.int32, device=dev)
        self.held, self.lens = ints([0] * batch), ints([0] * batch)
        # the trees
        seen = []
        for x, (up, _) in enumerate(TREE):
            seen.append((seen[up] if x else 0) | 1 << x)
        self.tree_mask = torch.tensor(seen * batch, dtype=torch.int64, device=dev).view(-1, 1)
        self.parents = ints([up for up, _ in TREE] * batch)
        self.depths = ints([bin(s).count("1") - 1 for s in seen] * batch)
        self.cu_q = ints([n * b for b in range(batch + 1)])
        # what each sequence holds in the cache (the prompt is not penalised), and its last token, which is not there yet
        self.history = torch.zeros(batch, most_new + n + 1, dtype=torch.int32, device=dev)
        self.history_lens, self.last = ints([0] * batch), torch.randint(0, vocab, (batch,), device=dev, generator=gen).int()
        self.repetition = 1 + 0.3 * torch.rand(batch, device=dev, generator=gen)
        self.frequency, self.presence = (0.2 * torch.rand(batch, device=dev, generator=gen) for _ in range(2))
        self.read_prompt(prompt)

    def gemv(self, weight, x, dtype=torch.bfloat16):
        """The fused GEMV in slabs of its widest batch."""
        return torch.cat([nf4.gemv(weight, x[i:i + 64], out_dtype=dtype) for i in range(0, x.shape[0], 64)])

    def heads(self, weight, x):
        return self.gemv(weight, x).view(x.shape[0], -1, self.dim)

    def read_prompt(self, tokens: torch.Tensor) -> None:
        x, at = self.embed[tokens], torch.arange(self.prompt, device=tokens.device)
        nf4.nf4_kv_append(self.k_cache, self.v_cache, at, self.heads(self.wk, x), self.heads(self.wv, x), at, self.cos_sin,
                          k_weight=self.k_norm)

    def step(self) -> None:
        """One tree of every sequence; history, lens and last move on. Nothing is read back, all state is kept in place."""
        n, b = len(TREE), self.batch
        draft = torch.empty(b, n, dtype=torch.int32, device=self.last.device)
        draft[:, 0] = self.last
        for level in LEVELS:
            for x in level:
                draft[:, x] = self.followers[draft[:, TREE[x][0]].long(), TREE[x][1]]
        tokens = draft.view(-1)
        slots, positions, lens, _, _ = nf4.nf4_kv_pages(
            self.lens, self.page_table, self.held, self.free_pages, self.free_count, PAGE, cu_q=self.cu_q, depths=self.depths,
            first_position=self.prompt, new_held=self.held, new_free_count=self.free_count)
        x = self.embed[tokens.long()]
        q = nf4.nf4_kv_append(self.k_cache, self.v_cache, slots, self.heads(self.wk, x), self.heads(self.wv, x), positions,
                              self.cos_sin, q=self.heads(self.wq, x), q_weight=self.q_norm, k_weight=self.k_norm)
        out = nf4.nf4_tree_attention(q, self.k_cache, self.v_cache, self.prefix_pages, self.prompt, self.page_table, lens,
                                     self.tree_mask, cu_q=self.cu_q)
        y = x + self.gemv(self.wo, out.view(b * n, -1))
        logits = self.gemv(self.head, y, torch.float32)
        _, best = nf4.nf4_adjust_logits(logits, history=self.history, history_lens=self.history_lens,
                                        repetition=self.repetition, frequency=self.frequency, presence=self.presence,
                                        cu_rows=self.cu_q, draft_tokens=tokens, tree_mask=self.tree_mask, out=logits,
                                        return_best=True)
        accepted, path, chosen, lens = nf4.nf4_tree_commit(self.parents, tokens, best, self.cu_q, lens, len(LEVELS) + 1,
                                                           page_table=self.page_table, k_cache=self.k_cache,
                                                           v_cache=self.v_cache)
        # the accepted nodes' tokens are in the cache now; what lies behind them goes to the spare last column
        j = torch.arange(path.shape[1], device=path.device)
        at = torch.where(j < accepted[:, None], self.history_lens[:, None] + j, self.history.shape[1] - 1)
        self.history.scatter_(1, at.clamp(max=self.history.shape[1] - 1), draft.gather(1, path.clamp(min=0).long()))
        self.history_lens += accepted
        self.lens.copy_(lens)
        self.last.copy_(chosen.gather(1, accepted[:, None].long() - 1)[:, 0])


def run(batch: int, prompt: int, steps: int, seed: int = 1):
    """Decodes `steps` trees per sequence; returns (decoder, prompt tokens, us per step)."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    tokens = torch.randint(0, 2000, (prompt,), device="cuda", generator=gen)
    d = TreeDecoder(batch, tokens, most_new=steps * (len(LEVELS) + 1), seed=seed)
    state = [t for t in vars(d).values() if isinstance(t, torch.Tensor)]
    before = [t.clone() for t in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.step()  # once outside the recording: modules load, allocations settle
        for t, s in zip(state, before):
            t.copy_(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            d.step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record(side)
        for _ in range(steps):
            graph.replay()
        end.record(side)
    side.synchronize()
    if nf4.nf4_device_error_flags() != 0:
        raise RuntimeError("device error flags set")
    return d, tokens, start.elapsed_time(end) * 1e3 / steps


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=32)
    args = ap.parse_args()
    d, _, us = run(args.batch, args.prompt, args.steps)
    per = float(d.history_lens.float().mean()) / args.steps
    print(f"{args.batch} sequences over a prompt of {args.prompt}: {us:.1f} us per step, {per:.2f} tokens per step and sequence")


if __name__ == "__main__":
    main()

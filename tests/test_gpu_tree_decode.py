"""The calls around a decode step as they are used together: examples/tree_decode.py (recorded steps of page tables,
append, attention of drafted trees, adjusted logits, and the accepted branch taken into the cache), against the same
model in binary64 torch from the tokens alone, one at a time.

Every token that was kept must be the best one by the model's logits, up to rounding. Tolerance: q, k and v, the
attention's weights and output and the o GEMV's output are rounded to bfloat16 (u = 2^-8) as in the test of
examples/shared_prefix_decode.py, so that the layer's output z is within 0.03 |z| in norm; y = x + z is rounded
once more; the head's GEMV is within 1e-3 of sum |w y|. A logit is w . y, so it moves by at most
|w| (0.03 |z| + u |y|) + 1e-3 sum |w| |y|, and the penalties stretch that by at most 1.3. A token may stand up to
twice that below the best."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("tree_decode", os.path.join(ROOT, "examples", "tree_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rotate(x, positions, base):
    half = x.shape[-1] // 2
    a = positions.double()[:, None] * base ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    p, r = x[..., :half], x[..., half:]
    return torch.cat((p * c - r * s, r * c + p * s), -1)


def norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()


@pytest.mark.parametrize("batch,prompt,steps", [(3, 40, 12), (9, 200, 7), (1, 1, 20)])
def test_kept_tokens_are_the_models(batch, prompt, steps):
    import w4a16_gemv_gb300 as nf4
    mod = example()
    d, tokens, _ = mod.run(batch, prompt, steps, seed=5)
    wq, wk, wv, wo, head = (nf4.dequant(w).view(w.shape).double() for w in (d.wq, d.wk, d.wv, d.wo, d.head))
    group, dim = d.q_heads // d.kv_heads, d.dim
    kept = d.history_lens.tolist()
    assert torch.equal(d.lens, d.history_lens) and min(kept) >= steps
    assert max(kept) > steps, "no drafted token was accepted"
    for b in range(batch):
        seq = torch.cat((d.history[b, :kept[b]], d.last[b:b + 1])).long()
        x = d.embed[torch.cat((tokens, seq[:-1]))].double()
        pos = torch.arange(x.shape[0], device="cuda")
        k = rotate(norm((x @ wk.T).view(-1, d.kv_heads, dim), d.k_norm), pos, 1e6).repeat_interleave(group, 1)
        v = (x @ wv.T).view(-1, d.kv_heads, dim).repeat_interleave(group, 1)
        q = rotate(norm((x @ wq.T).view(-1, d.q_heads, dim), d.q_norm), pos, 1e6)
        s = torch.einsum("thd,phd->htp", q, k) * dim ** -0.5
        s = s.masked_fill(pos[None, :] > pos[:, None], float("-inf"))
        z = torch.einsum("htp,phd->thd", torch.softmax(s, -1), v).reshape(x.shape[0], -1) @ wo.T
        y = x + z
        logits = y @ head.T
        tol = 1.3 * (head.norm(dim=1) * (0.03 * z.norm(dim=1) + 2.0 ** -8 * y.norm(dim=1))[:, None] +
                     1e-3 * (y.abs() @ head.abs().T))
        rho, f, p = (float(t[b]) for t in (d.repetition, d.frequency, d.presence))
        for i in range(kept[b]):  # after the i-th kept token came seq[i + 1]
            row = logits[prompt + i].clone()
            count = torch.bincount(seq[:i + 1], minlength=row.numel())
            known = count > 0
            row = torch.where(known, torch.where(row > 0, row / rho, row * rho) - f * count - p, row)
            best = int(row.argmax())
            short = float(row[best] - row[seq[i + 1]])
            assert short <= float(tol[prompt + i, best] + tol[prompt + i, seq[i + 1]]), (b, i, short)
    # every page once: in a row of the table, or free
    free = d.free_pages[:int(d.free_count)].tolist()
    rows = [d.page_table[b, :n].tolist() for b, n in enumerate(d.held.tolist())]
    assert sorted(free + [x for r in rows for x in r]) == list(range(-(-prompt // mod.PAGE), d.k_cache.shape[0]))


def test_two_recordings_share_nothing():
    """Two decoders, each with a graph of its own, replayed in turn on two streams: the results of each alone."""
    mod = example()
    alone = [mod.run(2, 30, 6, seed=s)[0] for s in (1, 2)]
    gen = torch.Generator(device="cuda")
    decoders, graphs, streams = [], [], []
    for s in (1, 2):
        gen.manual_seed(s + 1)
        d = mod.TreeDecoder(2, torch.randint(0, 2000, (30,), device="cuda", generator=gen), most_new=24, seed=s)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                d.step()
        decoders.append(d)
        graphs.append(g)
        streams.append(side)
    torch.cuda.synchronize()
    for _ in range(6):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, d in zip(alone, decoders):
        for name in ("history_lens", "lens", "last", "held", "free_count", "page_table"):
            assert torch.equal(getattr(a, name), getattr(d, name)), name
        n = int(a.history_lens.max())
        assert torch.equal(a.history[:, :n], d.history[:, :n])

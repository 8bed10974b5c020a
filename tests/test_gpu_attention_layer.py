"""The attention side of a decoder layer as it is used: examples/shared_prefix_decode.py (a prompt
appended once, then recorded steps of GEMV, append, attention, GEMV) against plain binary64 torch on
the dequantized weights.

Tolerance. Every stage rounds to bfloat16 (u = 2^-8): q, k and v after their GEMVs, q and k again after
the norm and rotation, the attention's weights and its output, and y. An error of relative size u in q or k
moves a score of size s by about u |s|, and so the weights by as much, relatively. With |s| below 4 sqrt(dim) ~ 45
in theory and about 4 here, the attention's output is within a few percent in the worst element and well under one
percent in norm: || y - y_exact || <= 0.03 || y_exact || per sequence and step."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    path = os.path.join(ROOT, "examples", "shared_prefix_decode.py")
    spec = importlib.util.spec_from_file_location("shared_prefix_decode", path)
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


@pytest.mark.parametrize("batch,prompt,steps", [(3, 100, 20), (20, 517, 5), (70, 33, 3)])
def test_layer(batch, prompt, steps):
    import w4a16_gemv_gb300 as nf4
    layer, x_prompt, xs, ys, _ = example().run(batch, prompt, steps, seed=7)
    wq, wk, wv, wo = (nf4.dequant(w).view(w.shape).double() for w in (layer.wq, layer.wk, layer.wv, layer.wo))
    group, dim = layer.q_heads // layer.kv_heads, layer.dim

    def keys_values(x, positions):
        x = x.double()
        k = (x @ wk.T).view(-1, layer.kv_heads, dim)
        return rotate(norm(k, layer.k_norm), positions, 1e6), (x @ wv.T).view(-1, layer.kv_heads, dim)
    kp, vp = keys_values(x_prompt, torch.arange(prompt, device="cuda"))
    own_k, own_v = [], []
    for i in range(steps):
        pos = torch.full((batch,), prompt + i, device="cuda")
        k, v = keys_values(xs[i], pos)
        own_k.append(k)
        own_v.append(v)
        q = rotate(norm((xs[i].double() @ wq.T).view(batch, layer.q_heads, dim), layer.q_norm), pos, 1e6)
        for b in range(batch):
            kb = torch.cat((kp, torch.stack([t[b] for t in own_k]))).repeat_interleave(group, 1)
            vb = torch.cat((vp, torch.stack([t[b] for t in own_v]))).repeat_interleave(group, 1)
            w = torch.softmax(torch.einsum("hd,phd->hp", q[b], kb) * dim ** -0.5, -1)
            y = torch.einsum("hp,phd->hd", w, vb).reshape(-1) @ wo.T
            err = float((ys[i, b].double() - y).norm() / y.norm())
            assert err <= 0.03, (i, b, err)

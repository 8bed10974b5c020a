"""Cases that measure the attention side of a decode step: the norm and rotation of queries and
keys, the append of keys and values to a paged cache, and attention over a cache whose first part
is shared by the whole batch.

``run`` computes them in plain torch operations (binary32, rounded once at the end), or, with
``own`` set, through this package's entry points. Head counts are those of the decoders that
bench.py names (12 query and 2 key/value heads, 32 and 32, of 128 elements) and generic ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6
BASE = 10000.0


# --------------------------------------------------------------------------------------- cases

def _rope(name, tokens, hq, hk, dim, rot, dtype, interleaved, norm, max_pos):
    return dict(name=name, op="qk_norm_rope", tokens=tokens, hq=hq, hk=hk, dim=dim, rot=rot, dtype=dtype,
                interleaved=interleaved, norm=norm, max_pos=max_pos)


def _append(name, tokens, hq, hk, dim, rot, dtype, interleaved, norm, max_pos, page, pad):
    return dict(name=name, op="kv_append", tokens=tokens, hq=hq, hk=hk, dim=dim, rot=rot, dtype=dtype,
                interleaved=interleaved, norm=norm, max_pos=max_pos, page=page, pad=pad)


def _attn(name, batch, max_q, hq, hk, dim, dtype, prefix, suffix, page):
    return dict(name=name, op="prefix_attention", batch=batch, max_q=max_q, hq=hq, hk=hk, dim=dim, dtype=dtype,
                prefix=prefix, suffix=suffix, page=page)


def listed():
    return [
        # one sequence's next token: a launch's latency
        _rope("rope token", 1, 12, 2, 128, 128, "bf16", False, True, 32768),
        # a long prompt, all heads rotated and normed
        _rope("rope prompt", 8192, 32, 32, 128, 128, "bf16", False, True, 32768),
        # an odd number of tokens, a quarter of the head rotated in neighbouring pairs, no norm
        _rope("rope partial", 1021, 16, 4, 64, 16, "fp16", True, False, 4096),
        # binary32 activations
        _rope("rope wide", 2500, 12, 2, 128, 128, "fp32", False, True, 8192),
        # a batch of sequences, one token each: what every layer of a decode step does
        _append("append tokens", 64, 12, 2, 128, 128, "bf16", False, False, 32768, 16, 0),
        # prompts packed into one call, a few of the tokens padding
        _append("append prompt", 8000, 32, 32, 128, 128, "bf16", False, True, 16384, 64, 25),
        # keys and values alone, odd sizes
        _append("append odd", 333, 0, 4, 64, 32, "fp16", True, False, 2048, 24, 7),
        # two sequences over a short system prompt: latency
        _attn("attention pair", 2, 1, 12, 2, 128, "bf16", 300, 60, 16),
        # a serving batch over one long system prompt
        _attn("attention batch", 32, 1, 12, 2, 128, "bf16", 8192, 500, 16),
        # as many key/value heads as query heads: the cache is the traffic
        _attn("attention heads", 64, 1, 32, 32, 128, "fp16", 2048, 250, 64),
        # many answers sampled from one very long document
        _attn("attention document", 16, 1, 12, 2, 128, "bf16", 131071, 300, 64),
        # several questions (prompts of their own) against one cached document
        _attn("attention prompts", 8, 512, 12, 2, 128, "bf16", 8190, 700, 32),
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm; above a few hundred no whole multiple of a tile (the listed cases have those)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v - (v > 256 and v % 256 == 0)))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e11 + w["flops"] / 5e13  # about the plain form's: several passes in binary32


def draw(rng):
    heads = [(12, 2, 128), (32, 32, 128), (32, 8, 128), (16, 4, 64), (8, 1, 128), (6, 6, 96), (10, 2, 80)]
    most = {op: max(_cost(c) for c in listed() if c["op"] == op)
            for op in ("qk_norm_rope", "kv_append", "prefix_attention")}
    while True:
        op = rng.choice(["qk_norm_rope", "kv_append", "prefix_attention", "prefix_attention"])
        hq, hk, dim = rng.choice(heads)
        if op != "prefix_attention":
            dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"] if op == "qk_norm_rope" else ["bf16", "fp16"])
            rot = rng.choice([dim, dim, dim // 2])
            c = dict(op=op, tokens=_log_int(rng, 1, 8192), hq=hq, hk=hk, dim=dim, rot=rot, dtype=dtype,
                     interleaved=rng.random() < 0.4, norm=rng.random() < 0.5, max_pos=_log_int(rng, 1000, 40000))
            if op == "kv_append":
                c.update(page=rng.choice([1, 16, 24, 64, 128]), pad=rng.choice([0, 0, 5]), hq=rng.choice([0, hq, hq]))
        else:
            c = dict(op=op, batch=_log_int(rng, 1, 128), max_q=rng.choice([1, 1, 1, _log_int(rng, 2, 512)]), hq=hq,
                     hk=hk, dim=dim, dtype=rng.choice(["bf16", "bf16", "fp16"]), prefix=_log_int(rng, 1, 131072),
                     suffix=_log_int(rng, 1, 2000), page=rng.choice([16, 24, 32, 64, 128]))
            c["suffix"] = max(c["suffix"], c["max_q"])
        if _cost(c) <= most[op]:
            return c


# ---------------------------------------------------------------------------------- the lengths

def _lengths(case):
    """Query tokens and own (suffix) keys of each sequence: ragged, the same for every seed."""
    n, s = [], []
    for b in range(case["batch"]):
        n.append(case["max_q"] - (b * 61) % (case["max_q"] // 2 + 1))
        s.append(max(n[-1], case["suffix"] - (b * 97) % (case["suffix"] // 2 + 1)))
    return n, s


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "prefix_attention":
        n, s = _lengths(case)
        tokens, hq, hk, dim = sum(n), case["hq"], case["hk"], case["dim"]
        keys = case["prefix"] + sum(s)
        pairs = sum(a * (case["prefix"] + b) - a * (a - 1) // 2 for a, b in zip(n, s))
        return {"bytes": 2 * keys * hk * dim * size + 2 * tokens * hq * dim * size + 4 * tokens * hq
                + 4 * (case["prefix"] + sum(s)) // case["page"], "flops": 4 * pairs * hq * dim}
    tokens, dim, rot = case["tokens"], case["dim"], case["rot"]
    table = 4 * rot * min(tokens, case["max_pos"])
    if case["op"] == "qk_norm_rope":
        rows = tokens * (case["hq"] + case["hk"])
        return {"bytes": 2 * rows * dim * size + table + 8 * tokens, "flops": rows * (3 * rot + 4 * dim * case["norm"])}
    rows = tokens * (case["hq"] + 2 * case["hk"])
    return {"bytes": 2 * rows * dim * size + table + 16 * tokens,
            "flops": tokens * (case["hq"] + case["hk"]) * (3 * rot + 4 * dim * case["norm"])}


# ---------------------------------------------------------------------------------- the inputs

def _table(max_pos, rot, dev):
    """(cos, sin) of position * BASE^(-2i/rot), as a program makes it once when it starts."""
    inv = BASE ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, device=dev, dtype=torch.float64)[:, None] * inv
    return torch.stack((a.cos(), a.sin()), -1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hk, dim = case["hq"], case["hk"], case["dim"]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen).to(dt)

    st = {"case": dict(case), "op": case["op"]}
    if case["op"] == "prefix_attention":
        n, s = _lengths(case)
        page, batch = case["page"], case["batch"]
        own_pages = [-(-v // page) for v in s]
        width, shared = max(own_pages), -(-case["prefix"] // page)
        pool = shared + sum(own_pages) + 3
        order = torch.randperm(pool, device=dev, generator=gen).to(torch.int32)
        st["prefix_pages"] = order[:shared].contiguous()
        pages = torch.zeros(batch, width, dtype=torch.int32, device=dev)
        at = shared
        for b, c in enumerate(own_pages):
            pages[b, :c] = order[at:at + c]
            at += c
        st["suffix_pages"] = pages
        st["suffix_lens"] = torch.tensor(s, dtype=torch.int32, device=dev)
        st["cu_q"] = torch.tensor([sum(n[:b]) for b in range(batch + 1)], dtype=torch.int32, device=dev)
        st["k_cache"], st["v_cache"] = normal(pool, page, hk, dim), normal(pool, page, hk, dim)
        st["q"] = normal(sum(n), hq, dim) * 1.5
        st["scale"] = dim ** -0.5
        return st
    tokens = case["tokens"]
    qkv = normal(tokens, hq + 2 * hk, dim)  # one projection's output: q, k and v are views of it
    st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    st["positions"] = torch.randint(0, case["max_pos"], (tokens,), device=dev, generator=gen)
    st["cos_sin"] = _table(case["max_pos"], case["rot"], dev)
    st["q_weight"] = (1 + 0.2 * torch.randn(dim, device=dev, generator=gen)).to(dt) if case["norm"] and hq else None
    st["k_weight"] = (1 + 0.2 * torch.randn(dim, device=dev, generator=gen)).to(dt) if case["norm"] else None
    if case["op"] == "kv_append":
        page = case["page"]
        pool = -(-tokens // page) + 5
        slots = torch.randperm(pool * page, device=dev, generator=gen)[:tokens]
        if case["pad"]:
            slots[torch.arange(tokens, device=dev) % (tokens // case["pad"] + 1) == 1] = -1
        st["slots"] = slots.contiguous()
        st["k_cache"], st["v_cache"] = normal(pool, page, hk, dim), normal(pool, page, hk, dim)
    return st


# ---------------------------------------------------------------------------------- the plain form

def _norm_rotate(x, weight, positions, cos_sin, interleaved):
    """[tokens, heads, dim] in binary32: each head's norm (with a weight), then the rotation."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    half = cos_sin.shape[1]
    cs = cos_sin[positions]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((turned, rest), -1)


def _plain_rope(st):
    il = st["case"]["interleaved"]
    return [_norm_rotate(st[n], st[n + "_weight"], st["positions"], st["cos_sin"], il).to(st[n].dtype) for n in "qk"]


def _plain_append(st):
    il, kc, vc, slots = st["case"]["interleaved"], st["k_cache"], st["v_cache"], st["slots"]
    k = _norm_rotate(st["k"], st["k_weight"], st["positions"], st["cos_sin"], il).to(kc.dtype)
    real = slots >= 0
    at = slots[real]
    kc.view(-1, *kc.shape[2:])[at] = k[real]
    vc.view(-1, *vc.shape[2:])[at] = st["v"][real]
    if not st["case"]["hq"]:
        return [kc, vc]
    return [_norm_rotate(st["q"], st["q_weight"], st["positions"], st["cos_sin"], il).to(st["q"].dtype), kc, vc]


def _part(scores, v):
    """Row maxima, sums and unscaled products of one part of the keys."""
    m = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return m, e.sum(-1, keepdim=True), e @ v


def _plain_attention(st):
    case, q = st["case"], st["q"]
    tokens, hq, dim = q.shape
    hk, batch, most = case["hk"], case["batch"], case["max_q"]
    group = hq // hk
    qf = q.float() * st["scale"]
    # the shared keys, once for all rows of a key/value head
    rows = qf.view(tokens, hk, group, dim).permute(1, 0, 2, 3).reshape(hk, tokens * group, dim)
    k, v = (st[n][st["prefix_pages"]].flatten(0, 1)[:case["prefix"]].permute(1, 0, 2).float()
            for n in ("k_cache", "v_cache"))
    m1, l1, o1 = (t.view(hk, tokens, group, -1) for t in _part(rows @ k.transpose(1, 2), v))
    # each sequence's own keys; its tokens padded to the longest
    cu, i = st["cu_q"].long(), torch.arange(most, device=q.device)
    n = cu[1:] - cu[:-1]
    own_rows = qf[(cu[:-1, None] + i).clamp(max=tokens - 1)].view(batch, most, hk, group, dim).transpose(1, 2)
    k, v = (st[t][st["suffix_pages"]].flatten(1, 2).permute(0, 2, 1, 3).float() for t in ("k_cache", "v_cache"))
    seen = torch.arange(k.shape[2], device=q.device) <= (st["suffix_lens"].long() - n)[:, None, None] + i[:, None]
    s2 = (own_rows.reshape(batch, hk, most * group, dim) @ k.transpose(2, 3)).view(batch, hk, most, group, -1)
    s2 = s2.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    of = torch.bucketize(torch.arange(tokens, device=q.device), cu[1:], right=True)
    at = torch.arange(tokens, device=q.device) - cu[of]
    m2, l2, o2 = (t.view(batch, hk, most, group, -1)[of, :, at].transpose(0, 1)
                  for t in _part(s2.view(batch, hk, most * group, -1), v))
    # both parts joined
    m = torch.maximum(m1, m2)
    a1, a2 = torch.exp(m1 - m), torch.exp(m2 - m)
    total = l1 * a1 + l2 * a2
    out = ((o1 * a1 + o2 * a2) / total).transpose(0, 1).reshape(tokens, hq, dim).to(q.dtype)
    return [out, (m + total.log())[..., 0].transpose(0, 1).reshape(tokens, hq)]


def run(st):
    if not own:
        return {"qk_norm_rope": _plain_rope, "kv_append": _plain_append, "prefix_attention": _plain_attention}[st["op"]](st)
    import w4a16_gemv_gb300 as nf4
    if st["op"] == "qk_norm_rope":
        return nf4.nf4_qk_norm_rope(st["q"], st["k"], st["positions"], st["cos_sin"], q_weight=st["q_weight"],
                                    k_weight=st["k_weight"], eps=EPS, interleaved=st["case"]["interleaved"])
    if st["op"] == "kv_append":
        q = nf4.nf4_kv_append(st["k_cache"], st["v_cache"], st["slots"], st["k"], st["v"], st["positions"],
                              st["cos_sin"], q=st["q"] if st["case"]["hq"] else None, q_weight=st["q_weight"],
                              k_weight=st["k_weight"], eps=EPS, interleaved=st["case"]["interleaved"])
        return [st["k_cache"], st["v_cache"]] if q is None else [q, st["k_cache"], st["v_cache"]]
    return nf4.nf4_prefix_attention(st["q"], st["k_cache"], st["v_cache"], st["prefix_pages"], st["case"]["prefix"],
                                    st["suffix_pages"], st["suffix_lens"], cu_q=st["cu_q"], scale=st["scale"],
                                    return_lse=True)


# ---------------------------------------------------------------------------------- 64 bits

def _exact_rows(x, weight, positions, rot, interleaved):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
    y = x.clone()
    for i in range(rot // 2):
        angle = positions.double() * BASE ** (-2.0 * i / rot)
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y[:, :, p] = x[:, :, p] * c - x[:, :, r] * s
        y[:, :, r] = x[:, :, r] * c + x[:, :, p] * s
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] != "prefix_attention":
        rows = {n: _exact_rows(st[n], st[n + "_weight"], st["positions"], case["rot"], case["interleaved"])
                for n in ("q", "k") if st[n].shape[1]}
        if case["op"] == "qk_norm_rope":
            return [rows["q"], rows["k"]]
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        for cache, new in ((kc, rows["k"]), (vc, st["v"].double())):
            keep = torch.nonzero(st["slots"] >= 0)[:, 0]
            where = st["slots"][keep]
            cache[where // case["page"], where % case["page"]] = new[keep]
        return ([rows["q"]] if case["hq"] else []) + [kc, vc]
    n, lens = _lengths(case)
    hq, hk, page = case["hq"], case["hk"], case["page"]
    tokens = sum(n)
    out = torch.empty(tokens, hq, case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.empty(tokens, hq, dtype=torch.float64, device="cuda")

    def keys(cache, table, count, head):
        j = torch.arange(count, device="cuda")
        return cache[table.long()[j // page], j % page, head].double()

    for head in range(hk):
        shared = [keys(st[c], st["prefix_pages"], case["prefix"], head) for c in ("k_cache", "v_cache")]
        qh = st["q"][:, head * (hq // hk):(head + 1) * (hq // hk)].double()
        step = max(1, 200_000_000 // (case["prefix"] * (hq // hk)))
        first = 0
        for b in range(case["batch"]):
            mine = [keys(st[c], st["suffix_pages"][b], lens[b], head) for c in ("k_cache", "v_cache")]
            k, v = (torch.cat(p) for p in zip(shared, mine))
            for t in range(first, first + n[b], step):
                u = min(t + step, first + n[b])
                sc = torch.einsum("tgd,pd->tgp", qh[t:u], k) * st["scale"]
                last = case["prefix"] + lens[b] - n[b] + torch.arange(t - first, u - first, device="cuda")
                sc[(torch.arange(k.shape[0], device="cuda") > last[:, None])[:, None].expand_as(sc)] = float("-inf")
                at = slice(head * (hq // hk), (head + 1) * (hq // hk))
                out[t:u, at] = torch.einsum("tgp,pd->tgd", torch.softmax(sc, -1), v)
                lse[t:u, at] = torch.logsumexp(sc, -1)
            first += n[b]
    return [out, lse]

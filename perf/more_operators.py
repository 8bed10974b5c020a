"""Cases that measure a step of speculative decoding beside its GEMVs: page tables and slots made from
the requests' lengths, attention of a tree of drafted tokens over the paged cache, penalties, biases
and grammar masks on logits, and taking the accepted branch of the tree into the cache.

``run`` computes them in plain torch operations (binary32, rounded once at the end), or, with ``own``
set, through this package's entry points. Head counts are those of the decoders that bench.py names
(12 query and 2 key/value heads, 32 and 32, of 128 elements) and generic ones; so are vocabularies.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BRANCH = 4     # children of a node: node x hangs on node (x - 1) // BRANCH
VOCAB = 32000  # of the drafted tokens where no logits are at hand


# --------------------------------------------------------------------------------------- cases

def _pages(name, batch, max_q, lens, page):
    return dict(name=name, op="kv_pages", batch=batch, max_q=max_q, lens=lens, page=page)


def _attn(name, batch, nodes, hq, hk, dim, dtype, prefix, suffix, page):
    return dict(name=name, op="tree_attention", batch=batch, nodes=nodes, hq=hq, hk=hk, dim=dim, dtype=dtype,
                prefix=prefix, suffix=suffix, page=page)


def _logits(name, batch, nodes, vocab, dtype, history, bias):
    return dict(name=name, op="adjust_logits", batch=batch, nodes=nodes, vocab=vocab, dtype=dtype, history=history,
                bias=bias)


def _commit(name, batch, nodes, layers, heads, dim, page):
    return dict(name=name, op="tree_commit", batch=batch, nodes=nodes, layers=layers, heads=heads, dim=dim, page=page)


def listed():
    return [
        # the next token of every sequence of a serving batch: a launch's latency
        _pages("pages tokens", 32, 1, 4000, 16),
        # prompts of many requests laid out in one call
        _pages("pages prompts", 256, 600, 2000, 16),
        # two sequences with a few drafted tokens each over a short system prompt: latency
        _attn("tree pair", 2, 8, 12, 2, 128, "bf16", 300, 60, 16),
        # a serving batch without a common prompt: the cache is the traffic
        _attn("tree batch", 16, 32, 32, 8, 128, "bf16", 0, 4000, 16),
        # one sequence with a very long context of its own
        _attn("tree long", 1, 25, 32, 32, 128, "bf16", 0, 50000, 64),
        # wide trees over one cached document
        _attn("tree document", 7, 64, 12, 2, 128, "bf16", 65000, 600, 32),
        # odd sizes: a page that ends inside a tile, a head that is no power of two
        _attn("tree odd", 37, 13, 10, 2, 80, "fp16", 777, 500, 24),
        # one sequence's next token over a small vocabulary of odd size: latency
        _logits("logits token", 1, 1, 32001, "fp32", 300, 10),
        # a serving batch, one token each, long answers
        _logits("logits batch", 64, 1, 128000, "bf16", 8000, 30),
        # every node of the batch's trees, each with its branch as context
        _logits("logits trees", 16, 32, 128000, "fp32", 3000, 30),
        # one layer's cache, a few sequences: latency
        _commit("commit layer", 4, 8, 1, 2, 128, 16),
        # all layers of a model at once
        _commit("commit layers", 64, 32, 28, 8, 128, 16),
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm; above a few hundred no whole multiple of a tile (the listed cases have those)."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v - (v > 256 and v % 256 == 0)))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6e11 + w["flops"] / 5e13  # about the plain form's: several passes in binary32


def draw(rng):
    ops = ("kv_pages", "tree_attention", "adjust_logits", "tree_commit")
    most = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ops}
    while True:
        op = rng.choice(ops + ("tree_attention",))
        if op == "kv_pages":
            c = dict(op=op, batch=_log_int(rng, 1, 300), max_q=rng.choice([1, _log_int(rng, 2, 64), _log_int(rng, 2, 600)]),
                     lens=_log_int(rng, 1, 20000), page=rng.choice([1, 16, 24, 64]))
            if c["batch"] * (c["lens"] + c["max_q"]) // c["page"] > 1 << 20:
                continue
        elif op == "tree_attention":
            hq, hk, dim = rng.choice([(12, 2, 128), (32, 32, 128), (32, 8, 128), (16, 4, 64), (8, 1, 128), (6, 6, 96),
                                      (10, 2, 80)])
            c = dict(op=op, batch=_log_int(rng, 1, 64), nodes=_log_int(rng, 1, 128), hq=hq, hk=hk, dim=dim,
                     dtype=rng.choice(["bf16", "bf16", "fp16"]), prefix=rng.choice([0, _log_int(rng, 1, 65536)]),
                     suffix=_log_int(rng, 1, 50000), page=rng.choice([16, 24, 32, 64, 128]))
            c["suffix"] = max(c["suffix"], c["nodes"])
            if c["batch"] * c["suffix"] * hk * dim > 64 * 4000 * 1024:  # keys in binary32 fit the card several times
                continue
        elif op == "adjust_logits":
            c = dict(op=op, batch=_log_int(rng, 1, 256), nodes=rng.choice([1, 1, _log_int(rng, 2, 64)]),
                     vocab=_log_int(rng, 1000, 260000), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                     history=_log_int(rng, 1, 40000), bias=rng.choice([0, 5, 100]))
        else:
            c = dict(op=op, batch=_log_int(rng, 1, 128), nodes=_log_int(rng, 1, 128), layers=_log_int(rng, 1, 40),
                     heads=rng.choice([1, 2, 8, 32]), dim=rng.choice([64, 80, 128]), page=rng.choice([1, 16, 24, 64]))
            if c["batch"] * 2 * c["nodes"] * c["layers"] * c["heads"] * c["dim"] > 1 << 30:
                continue
        if _cost(c) <= most[op]:
            return c


# ------------------------------------------------------------------- lengths and trees, the same for every seed

def _counts(most, batch):
    """Tokens or nodes of each sequence, ragged."""
    return [most - (b * 61) % (most // 2 + 1) for b in range(batch)]


def _own_lengths(case, n):
    """Own keys of each sequence with the drafted ones."""
    return [max(a, case["suffix"] - (b * 97) % (case["suffix"] // 2 + 1)) for b, a in enumerate(n)]


def _cached(case):
    """kv_pages: cached keys before the call, and pages held by then (some more, some fewer than needed)."""
    lens = [case["lens"] - (b * 97) % (case["lens"] // 2 + 1) for b in range(case["batch"])]
    held = [-(-v // case["page"]) + (2 if b % 5 == 3 else 0) for b, v in enumerate(lens)]
    return lens, held


def _path(n, b):
    """The branch that sequence b accepts: up to three nodes, the last child each time."""
    path = [0]
    while len(path) < 1 + b % 3:
        first = BRANCH * path[-1] + 1
        if first >= n:
            break
        path.append(min(first + BRANCH - 1, n - 1))
    return path


def _ancestors(nodes):
    """For each node of a tree its ancestors and itself, as lists."""
    rows = []
    for x in range(nodes):
        rows.append(([] if x == 0 else rows[(x - 1) // BRANCH]) + [x])
    return rows


def _tree_mask(counts, dev):
    """int64 [tokens, words]: bit x of token i's row is set where its context holds node x of its sequence's tree."""
    words = -(-max(counts) // 64)
    rows = []
    for r in _ancestors(max(counts)):
        w = [0] * words
        for x in r:
            w[x // 64] |= 1 << (x % 64)
        rows.append([v - (1 << 64) if v >> 63 else v for v in w])
    return torch.tensor([rows[i] for c in counts for i in range(c)], dtype=torch.int64, device=dev)


def work(case):
    op, batch = case["op"], case["batch"]
    if op == "kv_pages":
        n = _counts(case["max_q"], batch)
        lens, held = _cached(case)
        touched = sum(-(-(v + a) // case["page"]) - v // case["page"] for v, a in zip(lens, n))
        moved = sum(abs(-(-(v + a) // case["page"]) - h) for v, a, h in zip(lens, n, held))
        return {"bytes": 16 * sum(n) + 4 * touched + 8 * moved + 20 * batch, "flops": 0}
    n = _counts(case["nodes"], batch)
    if op == "tree_attention":
        s = _own_lengths(case, n)
        tokens, hq, hk, dim = sum(n), case["hq"], case["hk"], case["dim"]
        seen = [len(r) for r in _ancestors(max(n))]
        pairs = sum(a * (case["prefix"] + b - a) + sum(seen[:a]) for a, b in zip(n, s))
        keys = case["prefix"] + sum(s)
        return {"bytes": 4 * keys * hk * dim + 4 * tokens * hq * dim + 4 * tokens * hq + 4 * (keys // case["page"])
                + 8 * tokens * -(-max(n) // 64), "flops": 4 * pairs * hq * dim}
    if op == "adjust_logits":
        size = 4 if case["dtype"] == "fp32" else 2
        masked = sum(a for b, a in enumerate(n) if b % 3 != 2)
        return {"bytes": 2 * sum(n) * case["vocab"] * size + masked * case["vocab"] // 8 + 4 * sum(_histories(case))
                + 8 * case["bias"] * batch, "flops": 5 * sum(n) * case["vocab"]}
    rows = sum(sum(x != j for j, x in enumerate(_path(a, b))) for b, a in enumerate(n))
    return {"bytes": 8 * rows * case["layers"] * case["heads"] * case["dim"] + 12 * sum(n) + 40 * batch, "flops": 0}


def _histories(case):
    return [case["history"] - (b * 89) % (case["history"] // 2 + 1) for b in range(case["batch"])]


# ---------------------------------------------------------------------------------- the inputs

def _ints(values, dev, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=dev)


def _offsets(n, dev):
    return _ints([sum(n[:b]) for b in range(len(n) + 1)], dev)


def _table(order, at, counts, width):
    """Page tables [batch, width]: each sequence's pages, from order[at] on."""
    table = torch.zeros(len(counts), width, dtype=torch.int32, device=order.device)
    for b, c in enumerate(counts):
        table[b, :c] = order[at:at + c]
        at += c
    return table


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, batch = case["op"], case["batch"]

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, device=dev, generator=gen, dtype=torch.int32)

    st = {"case": dict(case), "op": op}
    if op == "kv_pages":
        n = _counts(case["max_q"], batch)
        lens, held = _cached(case)
        need = [-(-(v + a) // case["page"]) for v, a in zip(lens, n)]
        width = max(need + held) + 3
        pool = sum(need) + sum(held) + 7
        order = torch.randperm(pool, device=dev, generator=gen).to(torch.int32)
        st["page_table"] = _table(order, 0, held, width)
        free = pool - sum(held)  # the others, a stack: the last one is taken first
        st["free_pages"] = torch.cat((order[sum(held):], torch.full((sum(held),), -1, dtype=torch.int32, device=dev)))
        st["free_count"], st["lens"], st["held"] = _ints([free], dev), _ints(lens, dev), _ints(held, dev)
        st["cu_q"] = None if case["max_q"] == 1 else _offsets(n, dev)
        st["tokens"] = sum(n)
        return st
    n = _counts(case["nodes"], batch)
    tokens = sum(n)
    st["tree_mask"], st["cu_q"] = _tree_mask(n, dev), _offsets(n, dev)
    if op == "tree_attention":
        dt, hq, hk, dim, page = DTYPES[case["dtype"]], case["hq"], case["hk"], case["dim"], case["page"]

        def normal(*shape):
            return torch.randn(*shape, device=dev, generator=gen).to(dt)
        s = _own_lengths(case, n)
        own_pages, shared = [-(-v // page) for v in s], -(-case["prefix"] // page)
        pool = shared + sum(own_pages) + 3
        order = torch.randperm(pool, device=dev, generator=gen).to(torch.int32)
        st["prefix_pages"] = order[:shared].contiguous()
        st["suffix_pages"] = _table(order, shared, own_pages, max(own_pages))
        st["suffix_lens"] = _ints(s, dev)
        st["k_cache"], st["v_cache"] = normal(pool, page, hk, dim), normal(pool, page, hk, dim)
        st["q"] = normal(tokens, hq, dim) * 1.5
        st["scale"] = dim ** -0.5
        return st
    if op == "adjust_logits":
        vocab, h = case["vocab"], _histories(case)
        st["logits"] = (torch.randn(tokens, vocab, device=dev, generator=gen) * 3).to(DTYPES[case["dtype"]])
        # words come back: the history's tokens are spread over the logarithm of the vocabulary
        st["history"] = (vocab ** torch.rand(batch, max(h), device=dev, generator=gen)).int().clamp(0, vocab - 1)
        st["history_lens"], st["prompt_lens"] = _ints(h, dev), _ints([v // 3 for v in h], dev)
        for name, lo, hi in (("repetition", 1.0, 1.4), ("frequency", 0.0, 0.5), ("presence", 0.0, 0.8)):
            st[name] = lo + (hi - lo) * torch.rand(batch, device=dev, generator=gen)
        st["bias_tokens"] = ints(0, vocab, batch, case["bias"]) if case["bias"] else None
        st["bias_values"] = torch.randn(batch, case["bias"], device=dev, generator=gen) * 4 if case["bias"] else None
        if case["bias"]:
            st["bias_tokens"][:, case["bias"] * 2 // 3:] = torch.where(  # some requests have fewer
                torch.arange(batch, device=dev)[:, None] % 2 == 1, -1, st["bias_tokens"][:, case["bias"] * 2 // 3:])
        st["mask"] = torch.randint(-2 ** 31, 2 ** 31, (batch, -(-vocab // 32)), device=dev, generator=gen).to(torch.int32)
        st["mask_rows"] = _ints([-1 if b % 3 == 2 else b for b, c in enumerate(n) for _ in range(c)], dev)
        st["draft_tokens"] = (vocab ** torch.rand(tokens, device=dev, generator=gen)).int().clamp(0, vocab - 1)
        return st
    base = [40 + (b * 37) % 300 for b in range(batch)]  # cached keys before the drafted ones
    st["lens"] = _ints([v + a for v, a in zip(base, n)], dev)
    own_pages = [-(-(v + a) // case["page"]) for v, a in zip(base, n)]
    pool = sum(own_pages) + 2
    order = torch.randperm(pool, device=dev, generator=gen).to(torch.int32)
    st["page_table"] = _table(order, 0, own_pages, max(own_pages))
    st["parents"] = _ints([(x - 1) // BRANCH for c in n for x in range(c)], dev)
    start = ints(0, VOCAB, batch)
    of = torch.repeat_interleave(torch.arange(batch, device=dev), _ints(n, dev).long())
    node = torch.arange(tokens, device=dev) - st["cu_q"][:-1].long()[of]
    st["draft_tokens"] = ((start[of] + node) % VOCAB).to(torch.int32)  # no two of a tree alike
    st["targets"] = ints(VOCAB, 2 * VOCAB, tokens)                       # none of the drafted ones,
    chain = [_path(a, b) for b, a in enumerate(n)]                       # but along the accepted branch
    first = [sum(n[:b]) for b in range(batch)]
    at = [first[b] + x for b, p in enumerate(chain) for x in p[:-1]]
    to = [first[b] + x for b, p in enumerate(chain) for x in p[1:]]
    if at:
        st["targets"][_ints(at, dev).long()] = st["draft_tokens"][_ints(to, dev).long()]
    shape = (case["layers"], pool, case["page"], case["heads"], case["dim"])
    st["k_cache"], st["v_cache"] = (torch.randint(-30000, 30000, shape, device=dev, generator=gen, dtype=torch.int16)
                                    .to(torch.bfloat16) for _ in range(2))
    st["max_path"] = 8
    return st


# ---------------------------------------------------------------------------------- the plain form

def _plain_pages(st):
    page, table, stack, held = st["case"]["page"], st["page_table"], st["free_pages"], st["held"].long()
    dev, tokens, lens = table.device, st["tokens"], st["lens"].long()
    cu = torch.arange(lens.numel() + 1, device=dev) if st["cu_q"] is None else st["cu_q"].long()
    n = cu[1:] - cu[:-1]
    need = (lens + n + page - 1) // page
    col = torch.arange(table.shape[1], device=dev)
    # pages past the need go back, in order
    back = (col >= need[:, None]) & (col < held[:, None])
    count = st["free_count"].long()
    at = torch.where(back.flatten(), count + back.flatten().cumsum(0) - 1, stack.numel())
    stack.copy_(torch.cat((stack, stack[:1])).scatter_(0, at, table.flatten())[:-1])
    top = count + back.sum()
    # missing ones come from the top
    grow = (need - held).clamp(min=0)
    end = grow.cumsum(0)
    served = (end <= top) | (grow == 0)
    new = (col >= held[:, None]) & (col < need[:, None]) & served[:, None]
    k = (end - grow)[:, None] + col - held[:, None]
    table.copy_(torch.where(new, stack[(top - 1 - k).clamp(0, stack.numel() - 1)], table))
    t = torch.arange(tokens, device=dev)
    of = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    at = lens[of] + t - cu[of]
    slot = table[of, torch.where(served[of], at // page, 0)].long() * page + at % page
    return [torch.where(served[of], slot, -1), at, torch.where(served, lens + n, lens).int(),
            torch.where(served, need, held).int(), (top - torch.where(served, grow, 0).sum()).int(), table, stack]


def _part(scores, v):
    """Row maxima, sums and unscaled products of one part of the keys."""
    m = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return m, e.sum(-1, keepdim=True), e @ v


def _plain_attention(st):
    case, q = st["case"], st["q"]
    tokens, hq, dim = q.shape
    hk, batch, most = case["hk"], case["batch"], case["nodes"]
    group = hq // hk
    qf = q.float() * st["scale"]
    # each sequence's own keys; its tokens padded to the most
    cu, i = st["cu_q"].long(), torch.arange(most, device=q.device)
    n = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + i).clamp(max=tokens - 1)
    own_rows = qf[at].view(batch, most, hk, group, dim).transpose(1, 2)
    k, v = (st[t][st["suffix_pages"]].flatten(1, 2).permute(0, 2, 1, 3).float() for t in ("k_cache", "v_cache"))
    node = torch.arange(k.shape[2], device=q.device) - (st["suffix_lens"].long() - n)[:, None]  # of each key
    x = node.clamp(0, 64 * st["tree_mask"].shape[1] - 1)
    word = st["tree_mask"][at].gather(2, (x // 64)[:, None].expand(-1, most, -1))
    seen = ((word >> (x % 64)[:, None]) & 1).bool() & (node < n[:, None])[:, None] | (node < 0)[:, None]
    s2 = (own_rows.reshape(batch, hk, most * group, dim) @ k.transpose(2, 3)).view(batch, hk, most, group, -1)
    s2 = s2.masked_fill(~seen[:, None, :, None, :], float("-inf"))
    of = torch.bucketize(torch.arange(tokens, device=q.device), cu[1:], right=True)
    i = torch.arange(tokens, device=q.device) - cu[of]
    m, total, o = (t.view(batch, hk, most, group, -1)[of, :, i].transpose(0, 1)
                   for t in _part(s2.view(batch, hk, most * group, -1), v))
    if case["prefix"]:  # the shared keys, once for all rows of a key/value head, and both parts joined
        rows = qf.view(tokens, hk, group, dim).permute(1, 0, 2, 3).reshape(hk, tokens * group, dim)
        k, v = (st[t][st["prefix_pages"]].flatten(0, 1)[:case["prefix"]].permute(1, 0, 2).float()
                for t in ("k_cache", "v_cache"))
        m1, l1, o1 = (t.view(hk, tokens, group, -1) for t in _part(rows @ k.transpose(1, 2), v))
        m2 = m
        m = torch.maximum(m1, m2)
        a1, a2 = torch.exp(m1 - m), torch.exp(m2 - m)
        total, o = l1 * a1 + total * a2, o1 * a1 + o * a2
    out = (o / total).transpose(0, 1).reshape(tokens, hq, dim).to(q.dtype)
    return [out, (m + total.log())[..., 0].transpose(0, 1).reshape(tokens, hq)]


def _plain_logits(st):
    x = st["logits"].float()
    rows, vocab = x.shape
    dev, cu = x.device, st["cu_q"].long()
    r = torch.arange(rows, device=dev)
    of = torch.bucketize(r, cu[1:], right=True)
    # what stands in each request's prompt and answer, then on each row's branch
    col = torch.arange(st["history"].shape[1], device=dev)
    inside = col < st["history_lens"][:, None]
    h = st["history"].long()
    count = x.new_zeros(len(cu) - 1, vocab).scatter_add_(1, h, (inside & (col >= st["prompt_lens"][:, None])).float())
    seen = x.new_zeros(len(cu) - 1, vocab).scatter_add_(1, h, inside.float())
    count, seen = count[of], seen[of]
    for w in range(st["tree_mask"].shape[1]):
        for bit in range(min(64, st["case"]["nodes"] - 64 * w)):
            on = (st["tree_mask"][:, w] >> bit & 1).float()
            t = st["draft_tokens"][(cu[of] + 64 * w + bit).clamp(max=rows - 1)].long()
            count[r, t] += on
            seen[r, t] += on
    rho, f, p = (st[t][of][:, None] for t in ("repetition", "frequency", "presence"))
    x = torch.where(seen > 0, torch.where(x > 0, x / rho, x * rho), x)
    x = torch.where(count > 0, x - f * count - p, x)
    if st["bias_tokens"] is not None:
        t = st["bias_tokens"].long()
        bias = x.new_zeros(len(cu) - 1, vocab)
        for j in range(t.shape[1]):  # in the order of the list
            bias.scatter_add_(1, t[:, j:j + 1].clamp(min=0), torch.where(t >= 0, st["bias_values"], 0)[:, j:j + 1])
        x = x + bias[of]
    v = torch.arange(vocab, device=dev)
    bits = st["mask"][st["mask_rows"].clamp(min=0).long()][:, v // 32] >> (v % 32) & 1
    x = torch.where((bits == 0) & (st["mask_rows"] >= 0)[:, None], float("-inf"), x).to(st["logits"].dtype)
    top = x.amax(1, keepdim=True)
    return [x, torch.where(x == top, v, vocab).amin(1).int()]


def _plain_commit(st):
    cu, lens, page = st["cu_q"].long(), st["lens"].long(), st["case"]["page"]
    dev, batch, most = cu.device, len(cu) - 1, st["max_path"]
    n = cu[1:] - cu[:-1]
    tokens = st["parents"].numel()
    t = torch.arange(tokens, device=dev)
    of = torch.bucketize(t, cu[1:], right=True)
    x = t - cu[of]
    # the lowest child of each node that holds the model's choice there
    up = (cu[of] + st["parents"].long()).clamp(min=0)  # (the roots' own are not looked at)
    good = (x > 0) & (st["draft_tokens"] == st["targets"][up])
    after = torch.full((tokens,), tokens, device=dev).scatter_reduce_(0, up, torch.where(good, x, tokens), "amin")
    path, now = [torch.zeros(batch, dtype=torch.long, device=dev)], torch.zeros(batch, dtype=torch.long, device=dev)
    alive = n > 0
    steps = [alive]
    for _ in range(most - 1):
        nxt = after[(cu[:-1] + now).clamp(max=tokens - 1)]
        alive = alive & (nxt < tokens)
        now = torch.where(alive, nxt, now)
        path.append(now)
        steps.append(alive)
    path, steps = torch.stack(path, 1), torch.stack(steps, 1)
    accepted = steps.sum(1)
    chosen = st["targets"][cu[:-1, None] + path]
    j = torch.arange(most, device=dev)
    base = (lens - n)[:, None]

    def slot(key):
        key = torch.minimum(key, lens[:, None] - 1)
        return st["page_table"].gather(1, key // page).long() * page + key % page
    source = slot(base + path)
    place = torch.where(steps, slot(base + j), source)  # past the path: a row onto itself
    for c in (st["k_cache"], st["v_cache"]):
        rows = c.flatten(1, 2)
        keep = steps.flatten() & (path != j).flatten()
        moved = rows[:, torch.where(keep, source.flatten(), 0)]
        at = torch.where(keep, place.flatten(), rows.shape[1] - 1)  # no sequence has the pool's last page
        rows[:, at] = torch.where(keep[:, None, None], moved, rows[:, -1:])
    return [accepted.int(), torch.where(steps, path, -1).int(), torch.where(steps, chosen, -1).int(),
            (lens - n + accepted).int(), st["k_cache"], st["v_cache"]]


def run(st):
    if not own:
        return {"kv_pages": _plain_pages, "tree_attention": _plain_attention, "adjust_logits": _plain_logits,
                "tree_commit": _plain_commit}[st["op"]](st)
    import w4a16_gemv_gb300 as nf4
    if st["op"] == "kv_pages":
        made = nf4.nf4_kv_pages(st["lens"], st["page_table"], st["held"], st["free_pages"], st["free_count"],
                                st["case"]["page"], cu_q=st["cu_q"], tokens=st["tokens"])
        return [*made, st["page_table"], st["free_pages"]]
    if st["op"] == "tree_attention":
        return list(nf4.nf4_tree_attention(st["q"], st["k_cache"], st["v_cache"], st["prefix_pages"], st["case"]["prefix"],
                                           st["suffix_pages"], st["suffix_lens"], st["tree_mask"], cu_q=st["cu_q"],
                                           scale=st["scale"], return_lse=True))
    if st["op"] == "adjust_logits":
        return list(nf4.nf4_adjust_logits(
            st["logits"], history=st["history"], history_lens=st["history_lens"], prompt_lens=st["prompt_lens"],
            repetition=st["repetition"], frequency=st["frequency"], presence=st["presence"],
            bias_tokens=st["bias_tokens"], bias_values=st["bias_values"], mask=st["mask"], mask_rows=st["mask_rows"],
            cu_rows=st["cu_q"], draft_tokens=st["draft_tokens"], tree_mask=st["tree_mask"], return_best=True))
    made = nf4.nf4_tree_commit(st["parents"], st["draft_tokens"], st["targets"], st["cu_q"], st["lens"], st["max_path"],
                               page_table=st["page_table"], k_cache=st["k_cache"], v_cache=st["v_cache"])
    return [*made, st["k_cache"], st["v_cache"]]


# ---------------------------------------------------------------------------------- 64 bits

def _exact_pages(st, case):
    table, stack = st["page_table"].tolist(), st["free_pages"].tolist()
    n, (lens, held) = _counts(case["max_q"], case["batch"]), _cached(case)
    page, top = case["page"], int(st["free_count"])
    need = [-(-(v + a) // page) for v, a in zip(lens, n)]
    for b in range(len(n)):
        for c in range(need[b], held[b]):
            stack[top] = table[b][c]
            top += 1
    slots, positions, new_lens, new_held = [], [], [], []
    short = False
    for b in range(len(n)):
        more = max(need[b] - held[b], 0)
        short = short or more > top
        fits = more == 0 or not short
        if fits:
            for c in range(held[b], need[b]):
                top -= 1
                table[b][c] = stack[top]
        new_lens.append(lens[b] + n[b] if fits else lens[b])
        new_held.append(need[b] if fits else held[b])
        for key in range(lens[b], lens[b] + n[b]):
            slots.append(table[b][key // page] * page + key % page if fits else -1)
            positions.append(key)
    return [torch.tensor(v, dtype=d, device="cuda") for v, d in
            ((slots, torch.int64), (positions, torch.int64), (new_lens, torch.int32), (new_held, torch.int32),
             ([top], torch.int32), (table, torch.int32), (stack, torch.int32))]


def _exact_attention(st, case):
    n = _counts(case["nodes"], case["batch"])
    lens = _own_lengths(case, n)
    hq, hk, page = case["hq"], case["hk"], case["page"]
    group = hq // hk
    out = torch.empty(sum(n), hq, case["dim"], dtype=torch.float64, device="cuda")
    lse = torch.empty(sum(n), hq, dtype=torch.float64, device="cuda")
    branch = _ancestors(max(n))

    def keys(cache, table, count, head):
        j = torch.arange(count, device="cuda")
        return cache[table.long()[j // page], j % page, head].double()

    for head in range(hk):
        shared = [keys(st[c], st["prefix_pages"], case["prefix"], head) for c in ("k_cache", "v_cache")]
        at = slice(head * group, (head + 1) * group)
        first = 0
        for b in range(case["batch"]):
            mine = [keys(st[c], st["suffix_pages"][b], lens[b], head) for c in ("k_cache", "v_cache")]
            k, v = (torch.cat(p) for p in zip(shared, mine))
            hidden = torch.zeros(n[b], k.shape[0], dtype=torch.bool)
            hidden[:, -n[b]:] = True
            for i in range(n[b]):
                hidden[i, [case["prefix"] + lens[b] - n[b] + x for x in branch[i]]] = False
            rows = slice(first, first + n[b])
            sc = torch.einsum("tgd,pd->tgp", st["q"][rows, at].double(), k) * st["scale"]
            sc[hidden.cuda()[:, None].expand_as(sc)] = float("-inf")
            out[rows, at] = torch.einsum("tgp,pd->tgd", torch.softmax(sc, -1), v)
            lse[rows, at] = torch.logsumexp(sc, -1)
            first += n[b]
    return [out, lse]


def _exact_logits(st, case):
    n, h, vocab = _counts(case["nodes"], case["batch"]), _histories(case), case["vocab"]
    out = st["logits"].double()
    branch = _ancestors(max(n))
    first = 0
    v = torch.arange(vocab, device="cuda")
    for b in range(case["batch"]):
        rho, f, p = (float(st[t][b]) for t in ("repetition", "frequency", "presence"))
        words, start = st["history"][b, :h[b]].long(), h[b] // 3
        base_count = torch.bincount(words[start:], minlength=vocab)
        base_seen = torch.bincount(words, minlength=vocab)
        bias = torch.zeros(vocab, dtype=torch.float64, device="cuda")
        if case["bias"]:
            keep = st["bias_tokens"][b] >= 0
            bias.index_add_(0, st["bias_tokens"][b][keep].long(), st["bias_values"][b][keep].double())
        allowed = torch.ones(vocab, dtype=torch.bool, device="cuda")
        if b % 3 != 2:
            allowed = (torch.bitwise_and(st["mask"][b].long()[v // 32], 1 << (v % 32))) != 0
        for i in range(n[b]):
            extra = torch.bincount(st["draft_tokens"][[first + x for x in branch[i]]].long(), minlength=vocab)
            count, seen = base_count + extra, base_seen + extra
            x = out[first + i]
            x = torch.where(seen > 0, torch.where(x > 0, x / rho, x * rho), x)
            x = x - f * count.double() - p * (count > 0).double() + bias
            out[first + i] = x.masked_fill(~allowed, float("-inf"))
        first += n[b]
    # the best token of the rounded values: the first of the largest
    low = out.to(st["logits"].dtype)
    best = torch.stack([(row == row.max()).nonzero()[0, 0] for row in low])
    return [out, best.int()]


def _exact_commit(st, case):
    n = _counts(case["nodes"], case["batch"])
    parents, draft, targets = (st[t].tolist() for t in ("parents", "draft_tokens", "targets"))
    table, lens, page = st["page_table"].tolist(), st["lens"].tolist(), case["page"]
    k, v = st["k_cache"].clone(), st["v_cache"].clone()
    counts, paths, chosen, new_lens = [], [], [], []
    first = 0
    for b, a in enumerate(n):
        path = [0]
        while len(path) < st["max_path"]:
            fits = [x for x in range(1, a) if parents[first + x] == path[-1]
                    and draft[first + x] == targets[first + path[-1]]]
            if not fits:
                break
            path.append(fits[0])
        for j, x in enumerate(path):
            if x != j:
                to, at = lens[b] - a + j, lens[b] - a + x
                for new, old in ((k, st["k_cache"]), (v, st["v_cache"])):
                    new[:, table[b][to // page], to % page] = old[:, table[b][at // page], at % page]
        pad = [-1] * (st["max_path"] - len(path))
        counts.append(len(path))
        paths.append(path + pad)
        chosen.append([targets[first + x] for x in path] + pad)
        new_lens.append(lens[b] - a + len(path))
        first += a
    return [*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (counts, paths, chosen, new_lens)), k, v]


def exact(case, seed):
    st = prepare(case, seed)
    return {"kv_pages": _exact_pages, "tree_attention": _exact_attention, "adjust_logits": _exact_logits,
            "tree_commit": _exact_commit}[case["op"]](st, case)

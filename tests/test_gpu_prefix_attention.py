"""nf4_prefix_attention against softmax attention in binary64.

Tolerances. e = 2^-24, u the unit roundoff of the dtype. A score is a binary32 sum of D exact
products: within D e S of exact with S = scale * sum |q k| of the row's largest key; scaling it and
the exponential (2^-22 relative) add a few e, so a weight is within r = 2 e (D + 8) S + 16 e of exact,
relatively, and within u more once rounded for the product with v (fp16 also within 2^-25, its
subnormal step, of weights at most 1). Sums of N terms add N e. With A = sum p |v| and N the keys:
|out - exact| <= u |exact| + (u + 2 r + 2 N e) A + [fp16] 2^-24 sum |v| + tiny,
|lse - exact| <= r + N e + 4 e |exact|.
"""
import copy

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E = 2.0 ** -24


def lib():
    import w4a16_gemv_gb300 as nf4
    return nf4


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Call:
    """Inputs of one call. Slots of the caches that no token may see hold `junk`."""

    def __init__(self, hq, hk, dim, prefix, lens, counts, page=16, dt=torch.bfloat16, seed=0, junk=float("nan"),
                 heads_first=False, width=None, spread=1.0):
        g = gen(seed)
        self.hq, self.hk, self.dim, self.prefix, self.lens, self.counts, self.page = hq, hk, dim, prefix, lens, counts, page
        need = [-(-n // page) for n in lens]
        width = width if width is not None else max(need + [0])
        shared = -(-prefix // page)
        pool = shared + sum(need) + 2
        order = torch.randperm(pool, device="cuda", generator=g).int()
        self.prefix_pages = order[:shared].contiguous()
        self.suffix_pages = torch.full((len(lens), width), 1 << 30, dtype=torch.int32, device="cuda")
        at = shared
        for b, n in enumerate(need):
            self.suffix_pages[b, :n] = order[at:at + n]
            at += n
        self.suffix_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu_q = torch.tensor([sum(counts[:b]) for b in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
        shape = (pool, hk, page, dim) if heads_first else (pool, page, hk, dim)
        caches = [(torch.randn(shape, device="cuda", generator=g) * spread).to(dt) for _ in range(2)]
        self.k, self.v = (c.transpose(1, 2) if heads_first else c for c in caches)
        seen = torch.zeros(pool, page, dtype=torch.bool, device="cuda")
        for table, n in [(self.prefix_pages, prefix)] + [(self.suffix_pages[b], n) for b, n in enumerate(lens)]:
            j = torch.arange(n, device="cuda")
            seen[table[j // page].long(), j % page] = True
        self.k[~seen] = junk
        self.v[~seen] = junk
        self.q = (torch.randn(sum(counts), hq, dim, device="cuda", generator=g) * 1.5).to(dt)
        self.scale = dim ** -0.5

    def args(self):
        return (self.q, self.k, self.v, self.prefix_pages, self.prefix, self.suffix_pages, self.suffix_lens)

    def run(self, **kw):
        kw.setdefault("cu_q", self.cu_q)
        return lib().nf4_prefix_attention(*self.args(), scale=self.scale, return_lse=True, **kw)

    def rows(self, table, n):
        j = torch.arange(n, device="cuda")
        p = table[j // self.page].long()
        return self.k[p, j % self.page].double(), self.v[p, j % self.page].double()

    def check(self, got, what=""):
        out, lse = got
        u, g = U[out.dtype], self.hq // self.hk
        kp, vp = self.rows(self.prefix_pages, self.prefix)
        first = 0
        for b, n in enumerate(self.counts):
            ks, vs = self.rows(self.suffix_pages[b], self.lens[b])
            k = torch.cat((kp, ks)).repeat_interleave(g, 1)   # [keys, hq, dim]
            v = torch.cat((vp, vs)).repeat_interleave(g, 1)
            q = self.q[first:first + n].double()
            o, l = out[first:first + n].double(), lse[first:first + n].double()
            first += n
            if n == 0:
                continue
            keys = k.shape[0]
            s = torch.einsum("thd,phd->thp", q, k) * self.scale
            big = torch.einsum("thd,phd->thp", q.abs(), k.abs()) * self.scale
            last = self.prefix + self.lens[b] - n + torch.arange(n, device="cuda")
            j = torch.arange(keys, device="cuda")
            hidden = ((j > last[:, None]) & (j >= self.prefix))[:, None]  # the shared keys are seen by every token
            s, big = s.masked_fill(hidden, float("-inf")), big.masked_fill(hidden, 0.0)
            none = ((last < 0) & (self.prefix == 0))[:, None].expand(n, self.hq)
            assert (o[none] == 0).all() and (l[none] == float("-inf")).all(), f"{what}: rows without keys"
            if keys == 0:
                continue
            want_l = torch.logsumexp(s, -1)
            p = torch.exp(s - want_l[..., None]).masked_fill(none[..., None], 0.0)
            want = torch.einsum("thp,phd->thd", p, v)
            mass = torch.einsum("thp,phd->thd", p, v.abs())
            r = 2 * E * (self.dim + 8) * big.amax(-1) + 16 * E
            tol = u * want.abs() + (u + 2 * r + 2 * keys * E)[..., None] * mass + 1e-30
            if out.dtype == torch.float16:
                tol = tol + 2.0 ** -24 * torch.einsum("thp,phd->thd", (~hidden).double().expand_as(s), v.abs()) + 2.0 ** -24
            err = (o - want).abs()
            bad = ~(err <= tol) & ~none[..., None]
            assert not bad.any(), (f"{what}: sequence {b}: {int(bad.sum())} of {bad.numel()} outputs outside; worst "
                                   f"{float((err / tol).max()):.2f} x; first at {bad.nonzero()[0].tolist()}")
            bad = ~((l - want_l).abs() <= r + keys * E + 4 * E * want_l.abs()) & ~none
            assert not bad.any(), f"{what}: sequence {b}: lse outside"
        assert lib().nf4_device_error_flags() == 0, what


# ------------------------------------------------------------------------------------- decoding

@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("hq,hk,dim", [(12, 2, 128), (4, 4, 128), (7, 1, 128), (16, 4, 64), (10, 2, 80), (6, 6, 96),
                                       (2, 1, 8), (3, 3, 40)])
@pytest.mark.parametrize("prefix,batch", [(0, 3), (1, 1), (64, 2), (65, 5), (130, 33), (1000, 3), (3001, 40)])
def test_one_token_each(dt, hq, hk, dim, prefix, batch):
    lens = [1 + (b * 37 + prefix) % 150 for b in range(batch)]
    c = Call(hq, hk, dim, prefix, lens, [1] * batch, dt=dt, seed=prefix + batch)
    first = c.run()
    c.check(first, "cu_q")
    again = c.run(cu_q=None)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("page", [1, 2, 16, 24, 100, 256])
@pytest.mark.parametrize("heads_first", [False, True], ids=["slots-heads", "heads-slots"])
@pytest.mark.parametrize("batch", [2, 70])
def test_page_sizes_and_cache_orders(page, heads_first, batch):
    lens = [(b * 29) % 90 + 1 for b in range(batch)]
    c = Call(8, 2, 128, 777, lens, [1] * batch, page=page, heads_first=heads_first, seed=page)
    c.check(c.run())


@pytest.mark.parametrize("page", [8, 24, 40, 56, 72, 120, 136])
@pytest.mark.parametrize("hq,hk,dim", [(8, 2, 128), (3, 3, 64), (10, 2, 80)])
@pytest.mark.parametrize("prefix,counts,lens", [
    (1000, [1] * 40, [1 + 7 * b for b in range(40)]), (2641, [90, 160, 7], [90, 500, 333]), (119, [300], [480]),
    (0, [250, 130], [250, 401]), (6000, [70] * 3, [71, 120, 121])])
def test_pages_of_odd_multiples_of_eight(page, hq, hk, dim, prefix, counts, lens):
    c = Call(hq, hk, dim, prefix, lens, counts, page=page, seed=page + prefix)
    c.check(c.run())


@pytest.mark.parametrize("page", [12, 32])
@pytest.mark.parametrize("batch", [2, 70])
def test_keys_and_values_laid_out_apart(page, batch):
    """k as [pages, heads, slots, dim], v as a slice of a wider [pages, slots, heads, dim]."""
    c = Call(8, 2, 64, 300, [(b * 29) % 90 + 1 for b in range(batch)], [1] * batch, page=page, seed=18)
    want = c.run()
    c.k = c.k.transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.full((c.v.shape[0], page + 3, 4, 64), float("nan"), dtype=c.v.dtype, device="cuda")
    wide[:, 2:page + 2, 1:3] = c.v
    c.v = wide[:, 2:page + 2, 1:3]
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(got)


def test_one_cache_row_for_every_page():
    """Strides of zero: all pages, slots and heads share one row, so that the output is that row."""
    row = torch.randn(64, device="cuda").bfloat16()
    cache = row.expand(9, 16, 2, 64)
    q = torch.randn(40, 4, 64, device="cuda").bfloat16()
    table = torch.arange(4, dtype=torch.int32, device="cuda")
    own = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.tensor([17, 64], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3, 40], dtype=torch.int32, device="cuda")
    out = lib().nf4_prefix_attention(q, cache, cache, table, 60, own, lens, cu_q=cu)
    # sums of equal values: within the weights' rounding (2^-8) and the result's own
    assert ((out.double() - row.double()).abs() <= 2.0 ** -7 * row.double().abs() + 1e-30).all()


@pytest.mark.parametrize("prefix", [1, 2, 15, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1025])
@pytest.mark.parametrize("batch", [1, 30, 150])
def test_prefix_lengths_around_tiles(prefix, batch):
    c = Call(6, 2, 64, prefix, [b % 4 for b in range(batch)], [1] * batch, page=32, seed=prefix)
    # a sequence without own keys sees the prefix (its token is not in the cache yet)
    c.check(c.run())


# --------------------------------------------------------------------------- several tokens each

@pytest.mark.parametrize("hq,hk,dim", [(12, 2, 128), (4, 4, 128), (5, 1, 64), (6, 6, 96)])
@pytest.mark.parametrize("prefix,counts,lens", [
    (0, [5, 0, 1, 3], [5, 7, 1, 0]),            # no tokens, no keys, fewer keys than tokens
    (100, [3, 1, 2], [3, 50, 200]),
    (257, [130, 1, 0, 64, 65], [130, 9, 4, 70, 300]),
    (1000, [40] * 6, [40, 41, 60, 100, 39, 20]),  # the last two: some tokens see no own key
    (64, [300], [301]),
    (0, [200], [100]),                          # the first hundred rows see nothing
    (4000, [33, 700, 2], [33, 900, 1000]),
])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_ragged_tokens(dt, hq, hk, dim, prefix, counts, lens):
    c = Call(hq, hk, dim, prefix, lens, counts, dt=dt, seed=sum(counts) + prefix)
    c.check(c.run())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("hq,hk,dim", [(12, 2, 128), (4, 4, 64), (10, 2, 80)])
@pytest.mark.parametrize("prefix", [0, 1, 200, 700])
@pytest.mark.parametrize("counts,lens", [
    ([40, 0, 90, 13, 1], [40, 5, 300, 200, 1]),   # many rows per sequence
    ([300, 70], [0, 70]),                         # a sequence without keys of its own
    ([200, 100, 130], [150, 100, 700]),           # tokens before the first own key
    ([8] * 9, [8 + 11 * i for i in range(9)]), ([1] * 40, [i for i in range(40)])])
def test_tokens_that_no_sequence_holds(dt, hq, hk, dim, prefix, counts, lens):
    """Tokens before the first and after the last sequence see the shared keys only."""
    c = Call(hq, hk, dim, prefix, lens, counts, dt=dt, seed=prefix + len(lens), junk=0.0)
    c.check(c.run(), "all held")
    extra = (torch.randn(27, hq, dim, device="cuda", generator=gen(5)) * 1.5).to(dt)
    other = copy.copy(c)
    other.q, other.cu_q = torch.cat((extra[:7], c.q, extra[7:])), c.cu_q + 7
    out, lse = other.run()
    n = sum(counts)
    c.check((out[7:7 + n].contiguous(), lse[7:7 + n].contiguous()), "held")
    rest = copy.copy(c)
    rest.q, rest.counts, rest.lens = extra, [27], [0]
    rest.check(tuple(torch.cat((x[:7], x[7 + n:])) for x in (out, lse)), "not held")
    again = other.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_own_keys_alone_keep_infinities_out_of_rows_without_keys():
    """Without shared keys: a token before the first own key gives zeros whatever the keys hold."""
    for n, extra in ((3, 0), (9, 0), (100, 60)):
        c = Call(12, 2, 128, 0, [n - 2, n + 200], [n, n], seed=n)
        c.v[c.suffix_pages[0, 0].long(), 0] = float("inf")
        out, lse = c.run()
        assert not out[:2].any() and (lse[:2] == float("-inf")).all()
        assert out[2:n].isinf().all() and lib().nf4_device_error_flags() == 0
        out[2:n], lse[2:n] = 0, 0
        assert out[n:].isfinite().all()


def test_one_long_sequence_among_many():
    counts = [1] * 60 + [500] + [1] * 3
    lens = [10 + b for b in range(60)] + [700] + [5, 6, 1]
    c = Call(8, 2, 128, 300, lens, counts, seed=2)
    c.check(c.run())


def test_long_prefix():
    c = Call(12, 2, 128, 70001, [17, 200, 33], [1, 2, 1], page=64, seed=4)
    c.check(c.run())


def test_long_own_keys():
    c = Call(12, 2, 128, 10, [20000, 1, 300], [1, 1, 1], page=64, seed=5)
    c.check(c.run())


@pytest.mark.parametrize("spread", [0.02, 4.0, 30.0])
@pytest.mark.parametrize("batch", [2, 100])
def test_flat_and_sharp_weights(spread, batch):
    """Nearly equal weights, and rows that one key takes whole (scores of hundreds, growing along the keys)."""
    c = Call(8, 2, 128, 900, [50 + b for b in range(batch)], [1] * batch, spread=spread, seed=6, junk=float("inf"))
    ramp = torch.linspace(0.1, 1.0, c.k.shape[0], device="cuda")[:, None, None, None]
    c.k = (c.k.float() * ramp).nan_to_num(nan=float("nan"), posinf=float("inf")).to(c.k.dtype)
    c.check(c.run())


# -------------------------------------------------------------------------------- the interface

@pytest.mark.parametrize("junk", [float("nan"), float("inf"), float("-inf"), 3e38])
@pytest.mark.parametrize("batch", [3, 90])
def test_what_no_token_sees_does_not_matter(junk, batch):
    kw = dict(hq=8, hk=2, dim=128, prefix=333, lens=[(b * 31) % 70 + 1 for b in range(batch)],
              counts=[1 + b % 2 for b in range(batch)], page=48, seed=7)
    want = Call(junk=0.0, **kw).run()
    c = Call(junk=junk, **kw)
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(got)


def test_infinities_and_nan_that_are_seen():
    """A NaN key reaches every row of its head that sees it, and no other."""
    c = Call(4, 2, 64, 100, [20, 20], [1, 1], seed=8, junk=0.0)
    clean = c.run()
    j = 7
    c.k[c.suffix_pages[1, j // 16].long(), j % 16, 1, 3] = float("nan")
    out, lse = c.run()
    assert out[1, 2:].isnan().all() and lse[1, 2:].isnan().all()
    assert torch.equal(out[0], clean[0][0]) and torch.equal(out[1, :2], clean[0][1, :2])


@pytest.mark.parametrize("batch", [4, 64])
def test_strided_rows_and_given_outputs(batch):
    c = Call(6, 2, 64, 200, [9 + b for b in range(batch)], [1] * batch, seed=9)
    plain = c.run()
    qkv = torch.zeros(batch, 16, 64, dtype=c.q.dtype, device="cuda")
    qkv[:, 3:9] = c.q
    c.q = qkv[:, 3:9]
    buf = torch.full((batch, 9, 64), 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.empty(batch, 6, device="cuda")
    out = buf[:, 1:7]
    got = c.run(out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    assert (buf[:, 0] == 7).all() and (buf[:, 7:] == 7).all()
    only = lib().nf4_prefix_attention(*c.args(), cu_q=c.cu_q)
    assert torch.equal(only, plain[0])


def test_identical_calls_and_streams():
    c = Call(12, 2, 128, 5000, [100 + 7 * b for b in range(48)], [1] * 48, seed=10)
    want = c.run()
    torch.cuda.synchronize()
    nf4 = lib()
    need = nf4.nf4_prefix_attention_workspace_size(*c.args(), cu_q=c.cu_q)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # what it holds on entry does not matter
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        for kw in (dict(stream=s), dict(stream=s, workspace=ws), dict(stream=s.cuda_stream)):
            s.wait_stream(torch.cuda.current_stream())
            got = c.run(**kw)
            s.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with torch.cuda.stream(torch.cuda.Stream()):
        got = c.run()
        torch.cuda.current_stream().synchronize()
    assert torch.equal(got[0], want[0])
    with pytest.raises(nf4.NF4Error):
        c.run(workspace=ws[:need - 16])


@pytest.mark.parametrize("batch", [4, 40])
def test_recorded_graph_follows_growing_lengths(batch):
    """A graph recorded once serves every step: lengths are read on the device."""
    lens = [60 + b for b in range(batch)]
    c = Call(8, 2, 64, 500, lens, [1] * batch, page=16, seed=11, junk=0.25)
    out, lse = torch.empty_like(c.q), torch.empty(batch, 8, device="cuda")
    ws = torch.empty(lib().nf4_prefix_attention_workspace_size(*c.args(), cu_q=c.cu_q), dtype=torch.uint8, device="cuda")
    c.run(out=out, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, lse=lse, workspace=ws)
    for step in (1, 7, 40):
        c.lens = [(n * step) % 59 + 1 for n in lens]
        c.suffix_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check((out, lse), f"step {step}")


def test_indices_out_of_range():
    nf4 = lib()
    c = Call(4, 2, 64, 100, [20, 30, 10], [1, 2, 1], seed=12, junk=0.0)
    want = c.run()
    for bad in (-1, 1 << 20):  # a page of sequence 1: its rows are undefined, the others as they were
        keep = c.suffix_pages.clone()
        c.suffix_pages[1, 0] = bad
        got = c.run()
        assert nf4.nf4_device_error_flags() == 2
        assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][3], want[0][3])
        c.suffix_pages = keep
    for bad, as_if in ((-5, 0), (1 << 30, 32)):  # clamped to what the page table holds
        keep = c.suffix_lens.clone()
        c.suffix_lens[2] = bad
        c.suffix_pages[2, 1] = c.suffix_pages[0, 1]
        got = c.run()
        assert nf4.nf4_device_error_flags() == 2
        c.suffix_lens[2] = as_if
        ref = c.run()
        assert torch.equal(got[0], ref[0]) and nf4.nf4_device_error_flags() == 0
        c.suffix_lens = keep
    # cu_q past the tokens, and falling: nothing is read or written outside
    for cu in ([0, 1, 3, 9], [0, 3, 1, 4], [-4, 1, 3, 4]):
        c.run(cu_q=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert nf4.nf4_device_error_flags() == 2
    # tokens that no sequence holds attend to the prefix alone
    out, lse = c.run(cu_q=torch.tensor([0, 1, 3, 3], dtype=torch.int32, device="cuda"))
    alone = Call(4, 2, 64, 100, [20, 30, 10], [1, 2, 1], seed=12, junk=0.0)
    alone.suffix_lens.zero_()
    ref = alone.run()
    assert torch.equal(out[3], ref[0][3]) and torch.equal(lse[3], ref[1][3])


@pytest.mark.parametrize("batch,tokens", [(5, 5), (300, 700), (40, 3000)])
def test_any_cu_q(batch, tokens):
    """Whatever stands in cu_q, nothing outside the tensors is read or written."""
    nf4 = lib()
    g = gen(19)
    c = Call(6, 2, 64, 100, [1 + b % 40 for b in range(batch)], [0] * batch, seed=19, junk=0.0)
    q = torch.randn(tokens, 6, 64, device="cuda", generator=g).bfloat16()
    guard = torch.full((tokens + 2, 6, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    big = 2 ** 31 - 1
    for cu in (torch.randint(-10, tokens + 10, (batch + 1,), device="cuda", generator=g),
               torch.randint(-big, big, (batch + 1,), device="cuda", generator=g),
               torch.tensor([0, big], device="cuda").repeat(batch)[:batch + 1],
               torch.arange(batch + 1, device="cuda").flip(0)):
        nf4.nf4_prefix_attention(q, c.k, c.v, c.prefix_pages, 100, c.suffix_pages, c.suffix_lens, cu_q=cu.int(),
                                 out=guard[1:-1])
        torch.cuda.synchronize()
        assert (guard[0] == 7).all() and (guard[-1] == 7).all()
        assert nf4.nf4_device_error_flags() == 2


def test_cache_past_32_bits():
    """Pages whose offsets pass 2^32 elements."""
    page, hk, dim = 16, 2, 64
    stride = (1 << 31) + 128
    c = Call(4, hk, dim, 16, [16, 11], [1, 1], page=page, seed=13, junk=0.0)
    ref = c.run()
    ids = torch.cat((c.prefix_pages, c.suffix_pages[:, 0])).tolist()  # three pages: one shared, one of each sequence
    near = c.k, c.v
    far = [torch.empty(2 * stride + page * hk * dim, dtype=torch.bfloat16, device="cuda")
           .as_strided((3, page, hk, dim), (stride, hk * dim, dim, 1)) for _ in near]
    for new, old in enumerate(ids):
        for f, n in zip(far, near):
            f[new] = n[old]
    c.k, c.v = far
    c.prefix_pages = torch.tensor([0], dtype=torch.int32, device="cuda")
    c.suffix_pages = torch.tensor([[1], [2]], dtype=torch.int32, device="cuda")
    got = c.run()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_empty_calls():
    nf4 = lib()
    c = Call(4, 2, 64, 30, [], [], seed=15)
    assert c.run()[0].shape == (0, 4, 64)
    c = Call(4, 2, 64, 0, [0, 0], [1, 2], width=0)
    c.check(c.run())
    c = Call(4, 2, 64, 0, [0, 0], [1, 1], width=3)
    c.check(c.run())
    # an empty cache
    empty = torch.empty(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = nf4.nf4_prefix_attention(c.q, empty, empty, c.prefix_pages, 0, c.suffix_pages, c.suffix_lens,
                                        return_lse=True)
    assert (out == 0).all() and (lse == float("-inf")).all()
    # no batch: every token attends to the prefix alone
    c = Call(4, 2, 64, 30, [0], [3], width=0, seed=16)
    c.check(c.run())


def test_refusals_of_the_binding():
    nf4 = lib()
    c = Call(4, 2, 64, 30, [5, 6], [1, 1], seed=17)
    q, k, v, pp, p, sp, sl = c.args()
    with pytest.raises(TypeError):
        nf4.nf4_prefix_attention(q.half(), k, v, pp, p, sp, sl)
    with pytest.raises(TypeError):
        nf4.nf4_prefix_attention(q, k, v, pp.long(), p, sp, sl)
    with pytest.raises(ValueError):
        nf4.nf4_prefix_attention(q, k, v[:-1], pp, p, sp, sl)
    with pytest.raises(ValueError):
        nf4.nf4_prefix_attention(q, k, v, pp, 33, sp, sl)  # more keys than the pages hold
    with pytest.raises(ValueError):
        nf4.nf4_prefix_attention(q, k, v, pp, p, sp, sl[:1])
    with pytest.raises(ValueError):
        nf4.nf4_prefix_attention(q, k, v, pp, p, sp, sl, cu_q=c.cu_q[:2])
    with pytest.raises(ValueError):
        nf4.nf4_prefix_attention(q[..., :32], k, v, pp, p, sp, sl)
    with pytest.raises(ValueError):
        nf4.nf4_prefix_attention(q, k, v, pp, p, sp, sl, lse=torch.empty(2, 3, device="cuda"))
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_prefix_attention(q[:, :3], k, v, pp, p, sp, sl)  # 3 heads over 2
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_prefix_attention(q, k, v, pp, p, sp, sl, scale=-1.0)
    with pytest.raises(nf4.NF4Error):
        c2 = torch.empty(2 * 4 * 64 + 8, dtype=q.dtype, device="cuda")[1:].as_strided((2, 4, 64), (256, 64, 1))
        nf4.nf4_prefix_attention(c2, k, v, pp, p, sp, sl)

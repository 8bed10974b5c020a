"""nf4_tree_attention against softmax attention in binary64, and against nf4_prefix_attention where the
tree is a chain.

Tolerances. e = 2^-24, u the unit roundoff of the dtype (half a step: 2^-8 in bf16, 2^-11 in fp16). A score
is a binary32 sum of D exact products: within D e S of exact with S = scale * sum |q k| of the row's largest
key; scaling it and the exponential (2^-22 relative) add a few e, so a weight is within
r = 2 e (D + 8) S + 16 e of exact, relatively, and within u more once rounded for the product with v (fp16
also within 2^-25, its subnormal step, of weights at most 1). Sums of N terms add N e. With A = sum p |v|:
|out - exact| <= u |exact| + (u + 2 r + 2 N e) A + [fp16] 2^-24 sum |v| + tiny,
|lse - exact| <= r + N e + 4 e |exact|."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E = 2.0 ** -24


def lib():
    import w4a16_gemv_gb300 as nf4
    return nf4


def tree(rng, n, branch=3):
    """What each node of a random tree sees: its ancestors and itself."""
    seen = []
    for x in range(n):
        up = None if x == 0 else rng.randrange(max(0, (x - 1) // branch - 2), x)
        seen.append((set() if up is None else set(seen[up])) | {x})
    return seen


def words(seen, count, dev="cuda"):
    """The sets as int64 [tokens, count] words of bits."""
    rows = []
    for s in seen:
        w = [0] * count
        for x in s:
            if x < 64 * count:
                w[x // 64] |= 1 << (x % 64)
        rows.append([v - (1 << 64) if v >> 63 else v for v in w])
    return torch.tensor(rows, dtype=torch.int64, device=dev).view(len(seen), count)


class Call:
    """Inputs of one call; counts: nodes of each sequence, lens: own keys with them, seen: per token the set of nodes.
    Slots that no token may see hold NaN."""

    def __init__(self, hq, hk, dim, prefix, lens, counts, page=16, dt=torch.bfloat16, seed=0, seen=None, mask_words=None,
                 heads_first=False, width=None, behind=0):
        rng = random.Random(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
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
        caches = [torch.randn(shape, device="cuda", generator=g).to(dt) for _ in range(2)]
        self.k, self.v = (c.transpose(1, 2) if heads_first else c for c in caches)
        used = torch.zeros(pool, page, dtype=torch.bool, device="cuda")
        for table, n in [(self.prefix_pages, prefix)] + [(self.suffix_pages[b], n) for b, n in enumerate(lens)]:
            j = torch.arange(n, device="cuda")
            used[table[j // page].long(), j % page] = True
        self.k[~used] = float("nan")
        self.v[~used] = float("nan")
        self.seen = seen if seen is not None else [s for n in counts for s in tree(rng, n)]
        self.mask = words(self.seen + [set()] * behind, mask_words or -(-max(counts + [1]) // 64))
        self.q = (torch.randn(sum(counts) + behind, hq, dim, device="cuda", generator=g) * 1.5).to(dt)
        self.scale = dim ** -0.5

    def run(self, mask=None, **kw):
        kw.setdefault("cu_q", self.cu_q)
        return lib().nf4_tree_attention(self.q, self.k, self.v, self.prefix_pages, self.prefix, self.suffix_pages,
                                        self.suffix_lens, self.mask if mask is None else mask, scale=self.scale,
                                        return_lse=True, **kw)

    def rows(self, table, n):
        j = torch.arange(n, device="cuda")
        p = table[j // self.page].long()
        return self.k[p, j % self.page].double(), self.v[p, j % self.page].double()

    def hidden(self, b, first):
        """[tokens, keys]: what the sequence's tokens do not see."""
        n, length = self.counts[b], self.lens[b]
        h = torch.zeros(n, self.prefix + length, dtype=torch.bool)
        limit = 64 * self.mask.shape[1]
        for i in range(n):
            for x in range(max(0, n - length), n):
                h[i, self.prefix + length - n + x] = x not in self.seen[first + i] or x >= limit
        return h.cuda()

    def check(self, got, what=""):
        out, lse = got
        u, g = U[out.dtype], self.hq // self.hk
        kp, vp = self.rows(self.prefix_pages, self.prefix)
        first = 0
        for b, n in enumerate(self.counts):
            ks, vs = self.rows(self.suffix_pages[b], self.lens[b])
            k = torch.cat((kp, ks)).repeat_interleave(g, 1)
            v = torch.cat((vp, vs)).repeat_interleave(g, 1)
            q = self.q[first:first + n].double()
            o, l = out[first:first + n].double(), lse[first:first + n].double()
            if n == 0:
                continue
            hidden = self.hidden(b, first)[:, None]
            first += n
            keys = k.shape[0]
            none = hidden.all(-1).expand(n, self.hq) if keys else torch.ones(n, self.hq, dtype=torch.bool, device="cuda")
            assert (o[none] == 0).all() and (l[none] == float("-inf")).all(), f"{what}: rows without keys"
            if keys == 0:
                continue
            s = torch.einsum("thd,phd->thp", q, k) * self.scale
            big = torch.einsum("thd,phd->thp", q.abs(), k.abs()) * self.scale
            s, big = s.masked_fill(hidden, float("-inf")), big.masked_fill(hidden, 0.0)
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


HEADS = [(12, 2, 128), (4, 4, 128), (8, 1, 64), (10, 2, 80), (6, 6, 96), (2, 1, 8)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("hq,hk,dim", HEADS)
@pytest.mark.parametrize("prefix,counts,lens", [
    (0, [1], [1]), (0, [8, 3], [70, 3]), (300, [8, 5], [60, 41]), (0, [33, 1, 64, 20], [500, 64, 64, 130]),
    (1025, [13] * 9, [13 + 31 * b for b in range(9)]), (77, [0, 65, 2], [9, 200, 2]), (4000, [64, 128, 31], [64, 700, 1000]),
    (0, [200, 130], [1000, 130])])
def test_trees(dt, hq, hk, dim, prefix, counts, lens):
    c = Call(hq, hk, dim, prefix, lens, counts, dt=dt, seed=sum(counts) + prefix)
    got = c.run()
    c.check(got)
    again = c.run()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("hq,hk,dim", [(12, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("before", [0, 1, 15, 16, 17, 47, 63, 64, 65, 100, 120, 127, 128, 129, 190])
def test_nodes_at_every_offset_of_a_tile(hq, hk, dim, before):
    """Where a tile of keys, or a window of 64, begins within the nodes or before them."""
    for counts in ([5, 1], [40, 63], [150, 129]):
        c = Call(hq, hk, dim, 0, [n + before for n in counts], counts, seed=before)
        c.check(c.run(), str(counts))


@pytest.mark.parametrize("page", [1, 8, 24, 40, 56, 100, 256])
@pytest.mark.parametrize("heads_first", [False, True], ids=["slots-heads", "heads-slots"])
def test_page_sizes_and_cache_orders(page, heads_first):
    for counts in ([6, 3, 9], [100, 70]):
        lens = [n + 37 * (b + 1) for b, n in enumerate(counts)]
        c = Call(8, 2, 128, 333, lens, counts, page=page, heads_first=heads_first, seed=page)
        c.check(c.run(), str(counts))


@pytest.mark.parametrize("hq,hk,dim", [(12, 2, 128), (4, 4, 64), (3, 3, 40)])
@pytest.mark.parametrize("prefix", [0, 50])
@pytest.mark.parametrize("counts,lens", [([7, 20], [7, 90]), ([33] * 3, [33, 100, 64]), ([90, 160], [90, 400])])
def test_any_mask(hq, hk, dim, prefix, counts, lens):
    """Bits as they come: nodes that see nothing, not even themselves, or nodes behind them; bits past the nodes."""
    rng = random.Random(prefix + sum(lens))
    seen = []
    for n in counts:
        for i in range(n):
            kind = rng.randrange(4)
            seen.append(set() if kind == 0 else {rng.randrange(n)} if kind == 1 else
                        {x for x in range(n) if rng.random() < 0.5} if kind == 2 else set(range(n)))
    c = Call(hq, hk, dim, prefix, lens, counts, seed=prefix, seen=seen)
    got = c.run()
    c.check(got)
    mask = c.mask.clone()
    first = 0
    for n in counts:  # bits past a sequence's nodes are ignored
        for w in range(mask.shape[1]):
            past = sum(1 << x for x in range(64) if 64 * w + x >= n)
            mask[first:first + n, w] |= past - (1 << 64) if past >> 63 else past
        first += n
    again = c.run(mask=mask)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_rows_without_a_bit_see_nothing():
    for n in (4, 50, 200):
        c = Call(12, 2, 128, 0, [n, n + 3], [n, n], seen=[set()] * (2 * n), seed=n)
        out, lse = c.run()
        assert not out[:n].any() and (lse[:n] == float("-inf")).all()
        assert lse[n:].isfinite().all()
        c.check((out, lse))


@pytest.mark.parametrize("hq,hk,dim", [(12, 2, 128), (10, 2, 80), (4, 4, 64)])
@pytest.mark.parametrize("prefix,counts,lens", [
    (0, [5, 0, 1, 3], [5, 7, 1, 0]), (257, [130, 1, 0, 64], [130, 9, 4, 70]), (0, [200], [100]),
    (1000, [40] * 6, [40, 41, 60, 100, 39, 20]), (4000, [33, 300, 2], [33, 900, 1000])])
def test_a_chain_is_causal(hq, hk, dim, prefix, counts, lens):
    """Ones up to the own bit: what nf4_prefix_attention gives, within its tolerance, also where there are fewer keys
    than tokens."""
    c = Call(hq, hk, dim, prefix, lens, counts, seen=[set(range(i + 1)) for n in counts for i in range(n)], seed=prefix)
    got = c.run()
    c.check(got, "tree")
    want = lib().nf4_prefix_attention(c.q, c.k, c.v, c.prefix_pages, prefix, c.suffix_pages, c.suffix_lens, cu_q=c.cu_q,
                                      scale=c.scale, return_lse=True)
    c.check(want, "causal")
    assert torch.equal(got[1] == float("-inf"), want[1] == float("-inf"))


def test_one_token_each_without_offsets():
    lens = [1, 40, 200, 7]
    c = Call(8, 2, 128, 100, lens, [1] * 4, seed=4)
    a, b = c.run(), c.run(cu_q=None)
    c.check(a)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # a token that does not see itself
    blind = c.run(mask=torch.zeros_like(c.mask), cu_q=None)
    c.seen = [set()] * 4
    c.check(blind)


def test_fewer_words_than_nodes():
    """Nodes past the mask's bits are not seen."""
    for n in (100, 300):
        c = Call(6, 2, 64, 30, [n + 10], [n], mask_words=1, seed=n)
        c.check(c.run())


def test_mask_rows_apart_and_shared():
    c = Call(12, 2, 128, 0, [90, 50], [40, 8], seed=3)
    wide = torch.full((48, 5), -1, dtype=torch.int64, device="cuda")
    wide[:, 2:3] = c.mask
    got = c.run(mask=wide[:, 2:3])
    c.check(got)
    one = torch.tensor([[3]], dtype=torch.int64, device="cuda").expand(48, 1)  # every token sees nodes 0 and 1
    c.seen = [{0, 1}] * 48
    c.check(c.run(mask=one))


@pytest.mark.parametrize("counts", [[6, 9], [100, 70]])
def test_tokens_that_no_sequence_holds(counts):
    """Tokens before and behind the sequences see the shared keys only."""
    c = Call(12, 2, 128, 200, [n + 21 for n in counts], counts, seed=8)
    want = c.run()
    n = sum(counts)
    d = Call(12, 2, 128, 200, [m + 21 for m in counts], counts, seed=8, behind=9)
    d.q[4:4 + n] = c.q
    d.mask = torch.cat((d.mask[n:n + 4], c.mask, d.mask[n + 4:]))
    d.cu_q = c.cu_q + 4
    out, lse = d.run()
    c.check((out[4:4 + n].contiguous(), lse[4:4 + n].contiguous()))
    assert ((lse[4:4 + n] - want[1]).abs() <= 1e-4).all()
    alone = torch.cat((out[:4], out[4 + n:])), torch.cat((lse[:4], lse[4 + n:]))
    d.q, d.counts, d.lens, d.seen = torch.cat((d.q[:4], d.q[4 + n:])), [9], [0], [set()] * 9
    d.check(alone)


@pytest.mark.parametrize("counts,length", [([6, 9], 21), ([2, 3], 3000), ([100, 70], 21), ([64, 30], 5000), ([200, 130], 700)],
                         ids=str)
def test_tokens_that_no_sequence_holds_without_shared_keys(counts, length):
    """They see no key: zeros and -infinity."""
    c = Call(12, 2, 128, 0, [n + length for n in counts], counts, seed=8)
    want = c.run()
    c.check(want)
    n = sum(counts)
    d = Call(12, 2, 128, 0, [m + length for m in counts], counts, seed=8, behind=9)
    d.q[4:4 + n] = c.q
    d.mask = torch.cat((d.mask[n:n + 4], c.mask, d.mask[n + 4:]))
    d.cu_q = c.cu_q + 4
    out, lse = torch.full_like(d.q, 7.0), torch.full((n + 9, 12), 7.0, device="cuda")
    d.run(out=out, lse=lse)
    c.check((out[4:4 + n].contiguous(), lse[4:4 + n].contiguous()))
    assert not torch.cat((out[:4], out[4 + n:])).any()
    assert (torch.cat((lse[:4], lse[4 + n:])) == float("-inf")).all()


def test_infinities_in_keys_that_are_not_seen():
    """A key of infinities and NaN reaches the rows that see it alone."""
    for n in (6, 40, 150):
        seen = [{0, i} for i in range(n)]
        c = Call(12, 2, 128, 0, [n + 70], [n], seen=seen, seed=n)
        want = c.run()
        key = 70 + 3  # node 3's
        c.k[c.suffix_pages[0, key // 16].long(), key % 16] = float("nan")
        out, lse = c.run()
        rows = [i for i in range(n) if i != 3]
        assert torch.equal(out[rows], want[0][rows]) and torch.equal(lse[rows], want[1][rows])
        assert out[3].isnan().all() and lib().nf4_device_error_flags() == 0


def test_bad_lengths_pages_and_offsets_are_reported():
    c = Call(4, 2, 64, 0, [30, 20], [5, 3], seed=1)
    good = c.run()
    c.suffix_lens[0] = 10 ** 6  # more than the table holds
    c.run()
    assert lib().nf4_device_error_flags() == 2
    c.suffix_lens[0] = -1
    out, lse = c.run()
    assert lib().nf4_device_error_flags() == 2
    assert not out[:5].any() and torch.equal(out[5:], good[0][5:])
    c.suffix_lens[0] = 30
    c.cu_q[1] = 99
    c.run()
    assert lib().nf4_device_error_flags() == 2
    c.cu_q[1] = 5
    c.suffix_pages[1, 0] = -4
    out, _ = c.run()
    assert lib().nf4_device_error_flags() == 2 and torch.equal(out[:5], good[0][:5])


def test_recorded_and_replayed_as_sequences_grow():
    c = Call(12, 2, 128, 100, [20, 30], [8, 5], width=4, seed=2)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4) + int(c.k.shape[0])
    grown = [torch.cat((t, torch.randn(8, 16, 2, 128, device="cuda").bfloat16())) for t in (c.k, c.v)]
    for b in range(2):
        for i, p in enumerate(c.suffix_pages[b, :-(-c.lens[b] // 16)].long()):
            for t in grown:
                t[int(table[b, i])] = t[int(p)]
    c.k, c.v = grown
    c.k.nan_to_num_()
    c.v.nan_to_num_()
    c.suffix_pages = table
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, lse = c.run()
        for lens in ([20, 30], [33, 31], [64, 64]):
            c.suffix_lens.copy_(torch.tensor(lens))
            c.lens = lens
            graph.replay()
            c.check((out, lse), str(lens))
    side.synchronize()


@pytest.mark.parametrize("batch,nodes,length", [(1, 25, 40000), (3, 64, 9000), (2, 7, 70001)])
def test_long_caches(batch, nodes, length):
    for hq, hk, dim in ((8, 2, 128), (3, 3, 64)):
        c = Call(hq, hk, dim, 0, [length - 77 * b for b in range(batch)], [nodes] * batch, page=64, seed=length)
        c.check(c.run())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("hq,hk,dim", [(32, 8, 128), (16, 8, 64), (24, 8, 80)])
@pytest.mark.parametrize("page", [16, 24, 128])
@pytest.mark.parametrize("prefix", [0, 700])
def test_key_tiles_in_turns(dt, hq, hk, dim, page, prefix):
    """Up to 128 rows of a sequence over two key tiles and more: each half of the tiles has a softmax of its own."""
    lens = [129, 130, 200, 240, 241, 256, 257, 384, 385, 500, 640, 641, 900, 1024, 1025, 1150]
    c = Call(hq, hk, dim, prefix, lens, [1 + (7 * b) % 32 for b in range(16)], page=page, dt=dt, seed=page + prefix)
    c.check(c.run())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("hq,hk,dim", [(32, 8, 128), (16, 8, 64), (24, 8, 80)])
@pytest.mark.parametrize("page", [16, 24, 128])
@pytest.mark.parametrize("prefix", [8000, 8192, 12345])
@pytest.mark.parametrize("counts", [[8] * 4, [1, 31], [5, 0, 12, 7]], ids=str)
def test_shared_key_tiles_in_turns(dt, hq, hk, dim, page, prefix, counts):
    """Up to 128 rows of the whole call over a long shared prefix."""
    c = Call(hq, hk, dim, prefix, [n + 40 * b for b, n in enumerate(counts)], counts, page=page, dt=dt, seed=page + prefix)
    c.check(c.run())


@pytest.mark.parametrize("hk,dim", [(8, 64), (8, 128)])
@pytest.mark.parametrize("page", [16, 24])
def test_rows_that_see_one_half_of_the_keys(hk, dim, page):
    rng = random.Random(3)
    seen = [{rng.choice((0, 119, 120, 127, rng.randrange(128)))} if rng.random() < 0.8 else set() for _ in range(16 * 128)]
    c = Call(hk, hk, dim, 0, [128] * 16, [128] * 16, page=page, seed=page, seen=seen)
    c.check(c.run())


def test_infinities_and_nan_in_one_half_of_the_keys():
    c = Call(32, 8, 128, 0, [600] * 16, [30] * 16, seed=11)
    keys = c.k[c.suffix_pages[3, 590 // 16].long(), 590 % 16]  # a node that few rows see
    keys.fill_(float("nan"))
    out, lse = c.run()
    node, first = 590 - 570, 3 * 30
    hit = torch.tensor([node in c.seen[first + i] for i in range(30)], device="cuda")
    assert hit.any() and out[first:first + 30][hit].isnan().all() and not out[first:first + 30][~hit].isnan().any()
    rest = torch.ones(len(out), dtype=torch.bool, device="cuda")
    rest[first:first + 30] = False
    assert not out[rest].isnan().any() and not lse[rest].isnan().any()
    assert lib().nf4_device_error_flags() == 0


@pytest.mark.parametrize("prefix,counts,lens", [(300, [8, 5], [60, 41]), (0, [25] * 3, [700, 25, 3000]), (5000, [70, 9], [90, 200])])
def test_pages_past_32_bits(prefix, counts, lens):
    """Caches of 4.3 GB, whose last pages are the call's."""
    c = Call(12, 2, 128, prefix, lens, counts, seed=prefix)
    want = c.run()
    pages = 1 << 19
    pool = c.k.shape[0]
    big = torch.empty(2, pages, *c.k.shape[1:], dtype=c.k.dtype, device="cuda")
    big[0, -pool:], big[1, -pool:] = c.k, c.v
    c.k, c.v = big
    c.prefix_pages = c.prefix_pages + (pages - pool)
    c.suffix_pages = torch.where(c.suffix_pages < pool, c.suffix_pages + (pages - pool), c.suffix_pages)
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c.check(got)


@pytest.mark.parametrize("prefix", [0, 300, 8000])
def test_no_sequences_and_tables_of_no_columns(prefix):
    c = Call(12, 2, 128, prefix, [0, 0], [5, 3], seed=8, width=0)
    c.check(c.run())
    d = Call(12, 2, 128, prefix, [], [], seed=8, behind=9)
    out, lse = d.run()
    if prefix == 0:
        assert not out.any() and (lse == float("-inf")).all()
    d.counts, d.lens, d.seen = [9], [0], [set()] * 9
    d.suffix_pages = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    d.check((out, lse))


def test_the_last_word_of_the_widest_mask():
    """65536 nodes have a bit, the 70 behind them none: every row sees the last node that has one, row 5 the first too."""
    n = 65536 + 70
    c = Call(1, 1, 8, 0, [n], [n], seed=1, seen=[set()] * n, mask_words=1, page=64)
    mask = torch.zeros(n, 1024, dtype=torch.int64, device="cuda")
    mask[:, 1023], mask[5, 0] = -(1 << 63), 1
    out, lse = c.run(mask=mask)
    last = c.v[c.suffix_pages[0, 65535 // 64].long(), 65535 % 64, 0]
    same = (out[:, 0] == last).all(1)
    assert same[:5].all() and same[6:].all() and not same[5] and lib().nf4_device_error_flags() == 0


def test_two_streams_and_workspaces():
    c = Call(12, 2, 128, 2000, [300, 200], [9, 12], seed=5)
    want = c.run()
    args = (c.q, c.k, c.v, c.prefix_pages, c.prefix, c.suffix_pages, c.suffix_lens, c.mask)
    size = lib().nf4_tree_attention_workspace_size(*args, cu_q=c.cu_q)
    assert size > 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    got = [c.run(stream=s, workspace=w) for _ in range(5) for s, w in zip(streams, spaces)]
    torch.cuda.synchronize()
    assert all(torch.equal(g[0], want[0]) and torch.equal(g[1], want[1]) for g in got)
    with pytest.raises(lib().NF4Error, match="WORKSPACE"):
        c.run(workspace=spaces[0][:size - 1])


def test_refusals():
    c = Call(4, 2, 64, 0, [30, 20], [5, 3], seed=1)
    with pytest.raises(TypeError, match="int64"):
        c.run(mask=c.mask.int())
    with pytest.raises(ValueError, match="shape"):
        c.run(mask=c.mask[:7])
    with pytest.raises(ValueError, match="shape"):
        c.run(mask=c.mask[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        c.run(mask=c.mask.cpu())
    with pytest.raises(lib().NF4Error, match="INVALID_SIZE"):
        c.run(mask=c.mask[:, :0])

"""nf4_tree_commit against the same steps in plain Python. Rows are moved as they are: results are equal."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


def lib():
    import w4a16_gemv_gb300 as nf4
    return nf4


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def walk(parents, draft, targets, most):
    path = [0] if parents else []
    while path and len(path) < most:
        fits = [y for y in range(path[-1] + 1, len(parents)) if parents[y] == path[-1] and draft[y] == targets[path[-1]]]
        if not fits:
            break
        path.append(fits[0])
    return path


class Case:
    """counts: nodes of each sequence; chance: how likely a node's choice is one of its children."""

    def __init__(self, counts, seed=0, page=16, layers=None, heads=2, dim=64, dt=torch.bfloat16, chance=0.8, base=60,
                 heads_first=False, chain=False, offset=0):
        rng = random.Random(seed)
        self.counts, self.page = counts, page
        self.parents, self.draft, self.targets = [], [], []
        for n in counts:
            parents = [-1] + [x - 1 if chain else rng.randrange(max(0, x - 6), x) for x in range(1, n)]
            draft = [rng.randrange(50) for _ in range(n)]
            targets = [rng.randrange(100, 200) for _ in range(n)]
            for x in range(n):
                children = [y for y in range(x + 1, n) if parents[y] == x]
                if children and rng.random() < chance:
                    targets[x] = draft[rng.choice(children)]
            self.parents.append(parents[:n])
            self.draft.append(draft)
            self.targets.append(targets)
        self.base = [rng.randrange(base + 1) for _ in counts]
        self.lens = [a + n for a, n in zip(self.base, counts)]
        need = [-(-v // page) for v in self.lens]
        pool = sum(need) + 3
        order = list(range(pool))
        rng.shuffle(order)
        width = max(need + [1]) + 1
        self.table = [[1 << 29] * width for _ in counts]
        at = 0
        for b, c in enumerate(need):
            self.table[b][:c] = order[at:at + c]
            at += c
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        shape = (layers or 1, pool, heads, page, dim) if heads_first else (layers or 1, pool, page, heads, dim)
        self.k, self.v = (torch.randint(-2 ** 15, 2 ** 15, (*shape[:-1], dim + offset), device="cuda", generator=g,
                                        dtype=torch.int16).view(dt)[..., offset:] for _ in range(2))
        if heads_first:
            self.k, self.v = self.k.transpose(2, 3), self.v.transpose(2, 3)
        if layers is None:
            self.k, self.v = self.k[0], self.v[0]

    def flat(self, lists):
        return ints([x for s in lists for x in s])

    def args(self, most):
        cu = ints([sum(self.counts[:b]) for b in range(len(self.counts) + 1)])
        return self.flat(self.parents), self.flat(self.draft), self.flat(self.targets), cu, ints(self.lens), most

    def want(self, most):
        paths = [walk(p, d, t, most) for p, d, t in zip(self.parents, self.draft, self.targets)]
        k, v = self.k.clone(), self.v.clone()
        for b, path in enumerate(paths):
            for j, x in enumerate(path):
                at, to = ((self.table[b][i // self.page], i % self.page) for i in (self.base[b] + x, self.base[b] + j))
                for new, old in ((k, self.k), (v, self.v)):
                    if new.dim() == 5:
                        new[:, to[0], to[1]] = old[:, at[0], at[1]]
                    else:
                        new[to] = old[at]
        pad = [p + [-1] * (most - len(p)) for p in paths]
        chosen = [[self.targets[b][x] for x in p] + [-1] * (most - len(p)) for b, p in enumerate(paths)]
        return [len(p) for p in paths], pad, chosen, [a + len(p) for a, p in zip(self.base, paths)], k, v

    def kept(self, t, n):
        """The rows that a call leaves defined: everything but the rejected nodes' slots."""
        keep = torch.ones(t.shape[-4], self.page, dtype=torch.bool, device="cuda")
        for b, a in enumerate(n):
            for i in range(self.base[b] + a, self.lens[b]):
                keep[self.table[b][i // self.page], i % self.page] = False
        return t[..., keep, :, :] if t.dim() == 4 else t.flatten(1, 2)[:, keep.flatten()]

    def check(self, most, cache=True, **kw):
        n, path, chosen, lens, k, v = self.want(most)
        if cache:
            kw.update(page_table=ints(self.table), k_cache=self.k, v_cache=self.v)
        got = lib().nf4_tree_commit(*self.args(most), **kw)
        assert [g.tolist() for g in got] == [n, path, chosen, lens]
        if cache:
            for have, want in ((self.k, k), (self.v, v)):
                a, b = (self.kept(t, n).contiguous().view(torch.int16) for t in (have, want))
                assert torch.equal(a, b)
        assert lib().nf4_device_error_flags() == 0
        return got


@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("counts", [[1], [8, 3], [0, 5, 1, 40], [64, 33, 2] * 5, [500, 20], [9] * 130])
def test_trees(page, counts):
    for seed in range(3):
        Case(counts, seed=seed, page=page).check(16)
        Case(counts, seed=seed, page=page).check(16, cache=False)


@pytest.mark.parametrize("heads,dim", [(1, 64), (2, 128), (8, 128), (32, 80), (3, 20), (1, 7), (5, 512), (16, 1)])
@pytest.mark.parametrize("heads_first", [False, True], ids=["slots-heads", "heads-slots"])
@pytest.mark.parametrize("layers", [None, 1, 5])
def test_cache_shapes(heads, dim, heads_first, layers):
    Case([12, 30, 1], seed=dim, heads=heads, dim=dim, heads_first=heads_first, layers=layers, dt=torch.float16).check(8)
    Case([12, 30, 1], seed=dim, heads=heads, dim=dim, heads_first=heads_first, layers=layers, offset=3).check(8)


@pytest.mark.parametrize("n,most", [(2, 1024), (40, 1024), (40, 7), (40, 1), (1100, 1024), (1024, 1024), (4096, 1000)])
def test_chains(n, most):
    """Everything accepted: nothing moves; and a chain behind a rejected first child: every row moves by one."""
    c = Case([n, 3], seed=n, chain=True, chance=1.0)
    before = c.k.clone()
    got = c.check(most)
    assert int(got[0][0]) == min(n, most) and torch.equal(c.k.view(torch.int16), before.view(torch.int16))
    c = Case([n, 3], seed=n, chain=True, chance=1.0)
    c.parents[0] = [-1, 0] + [0 if x == 2 else x - 1 for x in range(2, n)]
    c.draft[0][0], c.draft[0][1] = 7, 8
    c.targets[0][0] = c.draft[0][2] if n > 2 else 500
    c.draft[0][1] = 900
    got = c.check(most)
    assert int(got[0][0]) == (min(n - 1, most) if n > 2 else 1)


def test_the_lowest_of_equal_children():
    c = Case([6], seed=1, chance=0.0)
    c.parents[0], c.draft[0], c.targets[0] = [-1, 0, 0, 0, 2, 3], [1, 5, 9, 9, 4, 4], [9, 0, 4, 4, 77, 0]
    got = c.check(6)
    assert got[1].tolist() == [[0, 2, 4, -1, -1, -1]] and got[2].tolist() == [[9, 4, 77, -1, -1, -1]]


def test_nodes_whose_parent_is_not_before_them():
    c = Case([5], seed=1, chance=0.0)
    for parents in ([0, 1, -3, 4, 9], [3, 0, 2, 1 << 30, -(1 << 31)]):
        draft, targets = [5] * 5, [5] * 5
        out = lib().nf4_tree_commit(ints(parents), ints(draft), ints(targets), ints([0, 5]), ints([9]), 5)
        want = walk([p if 0 <= p < x else -7 for x, p in enumerate(parents)], draft, targets, 5)
        assert out[0].tolist() == [len(want)] and out[1].tolist()[0][:len(want)] == want
        assert lib().nf4_device_error_flags() == 2
    # a node whose draft is no child's: its parent is not looked at beyond that
    assert lib().nf4_tree_commit(ints([12345]), ints([1]), ints([2]), ints([0, 1]), ints([9]), 5)[0].tolist() == [1]
    assert lib().nf4_device_error_flags() == 0


def test_bad_pages_lengths_and_offsets():
    def run(table=None, lens=None, cu=None):
        c = Case([6, 6], seed=3, chance=1.0, base=20)
        c.parents = [[-1, 0, 0, 2, 2, 4]] * 2
        c.draft, c.targets = [[0, 1, 2, 3, 4, 5]] * 2, [[2, 0, 4, 0, 5, 9]] * 2  # the path 0, 2, 4, 5
        a = list(c.args(8))
        if lens is not None:
            a[4] = ints(lens)
        if cu is not None:
            a[3] = ints(cu)
        before = c.k.clone(), c.v.clone()
        got = lib().nf4_tree_commit(*a, page_table=ints(c.table if table is None else table), k_cache=c.k, v_cache=c.v)
        same = torch.equal(c.k.view(torch.int16), before[0].view(torch.int16))
        return [g.tolist() for g in got], same, lib().nf4_device_error_flags()

    good, same, flags = run()
    assert good[0] == [4, 4] and not same and flags == 0
    for page in (-1, 1 << 30):
        out, same, flags = run(table=[[page] * 4] * 2)
        assert out == good and same and flags == 2
    assert run(lens=[2, -5])[2] == 2
    assert run(lens=[2 ** 31 - 1] * 2)[1:] == (True, 2)
    out, _, flags = run(cu=[0, 6, 99])
    assert flags == 2 and out[0] == [4, 4]
    out, _, flags = run(cu=[0, 99, 6])
    assert flags == 2 and out[0][1] == 0
    n = 4100  # nodes past the first 4096 are on no path
    out = lib().nf4_tree_commit(ints([x - 1 for x in range(n)]), ints([3] * n), ints([3] * n), ints([0, n]), ints([n]), 9)
    assert out[0].tolist() == [9] and lib().nf4_device_error_flags() == 2


def test_without_offsets_and_in_place():
    lens = ints([7, 1, 30])
    out = lib().nf4_tree_commit(ints([0, 0, 0]), ints([1, 2, 3]), ints([4, 5, 6]), None, lens, 2, new_lens=lens)
    assert [o.tolist() for o in out] == [[1, 1, 1], [[0, -1]] * 3, [[4, -1], [5, -1], [6, -1]], [7, 1, 30]]
    none = ints([])
    out = lib().nf4_tree_commit(none, none, none, ints([0, 0]), ints([5]), 2)
    assert [o.tolist() for o in out] == [[0], [[-1, -1]], [[-1, -1]], [5]]
    out = lib().nf4_tree_commit(none, none, none, None, none, 2)
    assert [o.tolist() for o in out] == [[], [], [], []]


def test_recorded_and_replayed():
    c = Case([20, 33], seed=4, layers=3)
    parents, draft, targets, cu, lens, most = c.args(8)
    table = ints(c.table)
    keep = c.k.clone(), c.v.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = lib().nf4_tree_commit(parents, draft, targets, cu, lens, most, page_table=table, k_cache=c.k, v_cache=c.v)
        for seed in (5, 6):
            d = Case([20, 33], seed=seed)
            c.parents, c.draft, c.targets = d.parents, d.draft, d.targets
            for t, s in ((parents, c.parents), (draft, c.draft), (targets, c.targets)):
                t.copy_(c.flat(s))
            c.k.copy_(keep[0])
            c.v.copy_(keep[1])
            n, path, chosen, new_lens, k, v = c.want(most)
            graph.replay()
            assert [o.tolist() for o in out] == [n, path, chosen, new_lens]
            for have, want in ((c.k, k), (c.v, v)):
                assert torch.equal(c.kept(have, n).view(torch.int16), c.kept(want, n).view(torch.int16))
    side.synchronize()


def test_refusals():
    c = Case([4, 3], seed=1)
    a = c.args(4)
    run = lib().nf4_tree_commit
    table = ints(c.table)
    with pytest.raises(TypeError, match="together"):
        run(*a, k_cache=c.k, v_cache=c.v)
    with pytest.raises(TypeError, match="together"):
        run(*a, page_table=table, k_cache=c.k)
    with pytest.raises(ValueError, match="shape"):
        run(*a, page_table=table, k_cache=c.k, v_cache=c.v[:2])
    with pytest.raises(TypeError, match="bf16 or fp16"):
        run(*a, page_table=table, k_cache=c.k.float(), v_cache=c.v.float())
    with pytest.raises(ValueError, match="max_path"):
        run(*a[:5], 0)
    with pytest.raises(TypeError, match="int32"):
        run(a[0], a[1], a[2].long(), *a[3:])
    with pytest.raises(lib().NF4Error, match="INVALID_SIZE"):
        run(*a, page_table=table, k_cache=c.k, v_cache=c.v, new_lens=a[4])
    with pytest.raises(lib().NF4Error, match="INVALID_SIZE"):
        run(a[0], a[1], a[2], None, a[4], 4)


@pytest.mark.parametrize("cache", [False, True], ids=["tokens", "cache"])
def test_fewer_keys_than_nodes_are_reported(cache):
    """The first nodes then have no key: new_lens is lens - n + accepted, at least 0, and the sequence is reported, also
    where nothing moves."""
    for lens, accepted in (([2, 20], 6), ([5, 6], 6), ([0, 9], 6), ([2, 20], 1)):
        c = Case([6, 6], seed=3, chain=True, chance=1.0, base=20)
        for t in c.targets:
            t[0] = t[0] if accepted == 6 else 777
        a = list(c.args(8))
        a[4] = ints(lens)
        kw = dict(page_table=ints(c.table), k_cache=c.k, v_cache=c.v) if cache else {}
        before = c.k.clone(), c.v.clone()
        got = lib().nf4_tree_commit(*a, **kw)
        assert got[0].tolist() == [accepted] * 2
        assert got[3].tolist() == [max(0, n - 6 + accepted) for n in lens]
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip((c.k, c.v), before))
        assert lib().nf4_device_error_flags() == 2, lens
        a[4] = ints([6, 20])
        lib().nf4_tree_commit(*a, **kw)
        assert lib().nf4_device_error_flags() == 0


def test_tables_without_a_page():
    """A table of no columns holds no row: what would move stays, and is reported; where nothing moves, nothing is."""
    for moves in (True, False):
        c = Case([6, 6], seed=3, chain=True, chance=1.0, base=20)
        if moves:
            c.parents = [[-1, 0, 0, 2, 2, 4]] * 2
            c.draft, c.targets = [[0, 1, 2, 3, 4, 5]] * 2, [[2, 0, 4, 0, 5, 9]] * 2
        before = c.k.clone(), c.v.clone()
        got = lib().nf4_tree_commit(*c.args(8), page_table=ints([]).view(2, 0), k_cache=c.k, v_cache=c.v)
        assert got[0].tolist() == ([4, 4] if moves else [6, 6])
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip((c.k, c.v), before))
        assert lib().nf4_device_error_flags() == (2 if moves else 0)


def one_buffer(shape, dt=torch.bfloat16):
    return torch.randint(-2 ** 15, 2 ** 15, shape, device="cuda", dtype=torch.int16).view(dt)


def test_caches_of_one_buffer():
    """Keys and values side by side, whichever dimension divides them, in one buffer."""
    base = Case([12, 30, 1], seed=7, layers=3)
    layers, pool, page, heads, dim = base.k.shape
    sides = [one_buffer((2, *base.k.shape)).unbind(0), one_buffer((layers, 2, *base.k.shape[1:])).unbind(1),
             one_buffer((layers, pool, 2, page, heads, dim)).unbind(2),
             one_buffer((layers, pool, page, 2, heads, dim)).unbind(3), one_buffer((layers, pool, page, heads, 2, dim)).unbind(4),
             one_buffer((layers, pool, page, heads, 2 * dim)).split(dim, -1),
             one_buffer((pool, 2, layers, page, heads, dim)).transpose(0, 2).unbind(1)]
    other = one_buffer((layers, 2, pool * page * heads * dim))  # the layers alike, the heads of one in front of its slots
    sides.append((other[:, 0].view(base.k.shape), other[:, 1].view(layers, pool, heads, page, dim).transpose(2, 3)))
    for k, v in sides:
        for first, second in ((k, v), (v, k)):
            c = Case([12, 30, 1], seed=7, layers=3)
            c.k, c.v = first, second
            c.check(8)


def test_caches_that_overlap_are_refused():
    c = Case([12, 30, 1], seed=7, layers=3)
    layers, pool, page, heads, dim = c.k.shape
    args, table = c.args(8), ints(c.table)
    wide = one_buffer((layers + 1, pool + 1, page, heads, 2 * dim))
    flat = one_buffer((layers * pool * page * heads * dim + 64,))

    def shifted(by):
        return flat[by:by + 64 * (flat.numel() // 64 - 1)].view(c.k.shape)
    pairs = [(c.k, c.k), (c.k, c.v[:, :, :, :1].expand_as(c.k)), (c.k[:1].expand_as(c.k), c.v),
             (c.k[:, :1].expand_as(c.k), c.v), (c.k[:, :, :1].expand_as(c.k), c.v),
             (wide[:layers, :pool, ..., :dim], wide[:layers, :pool, ..., dim - 1:2 * dim - 1]),
             (wide[:layers, :pool, ..., :dim], wide[:layers, 1:, ..., :dim]), (wide[:layers, :pool, ..., :dim], wide[1:, :pool, ..., :dim]),
             (shifted(0), shifted(1)), (shifted(64), shifted(0)),
             (flat.as_strided(c.k.shape, (pool * page * heads * dim // 2, page * heads * dim, heads * dim, dim, 1)), c.v),
             (wide[:layers, :pool, ..., :dim], wide[1:, 1:, ..., :dim])]
    for i, (k, v) in enumerate(pairs):
        before = k.clone(), v.clone()
        with pytest.raises((ValueError, lib().NF4Error), match="overlap|INVALID_SIZE"):
            lib().nf4_tree_commit(*args, page_table=table, k_cache=k, v_cache=v)
        assert torch.equal(k.view(torch.int16), before[0].view(torch.int16)), i
        assert torch.equal(v.view(torch.int16), before[1].view(torch.int16)), i
    # of a dimension of one element the stride says nothing
    one = Case([12, 30], seed=7, heads=1, layers=1)
    one.k = one.k.as_strided(one.k.shape, (0, *one.k.stride()[1:3], 0, 1))
    one.check(8)


def moving(c, moves):
    """Gives sequence b a tree whose accepted branch lies moves[b] rows (of moves[b] + 2 nodes) behind a rejected first
    child: all of its nodes but node 0 move by one."""
    for b, m in enumerate(moves):
        n = c.counts[b]
        assert n == m + 2
        c.parents[b] = [-1, 0] + [0 if x == 2 else x - 1 for x in range(2, n)]
        c.draft[b] = [900 + x for x in range(n)]
        c.targets[b] = [c.draft[b][x + 1] for x in range(n - 1)] + [7]
        if n > 2:
            c.targets[b][0] = c.draft[b][2]
        else:
            c.targets[b][0] = 7
    return c


@pytest.mark.parametrize("batch,heads,dim,layers", [(130, 8, 128, 7), (300, 2, 64, 7), (460, 1, 64, 9), (1000, 1, 20, 3)])
@pytest.mark.parametrize("moves", [[1], [3], [8], [9], [0, 1, 3, 8, 9, 17, 5]], ids=str)
def test_blocks_of_several_layers(batch, heads, dim, layers, moves):
    """More sequences than there are places for a block of each layer (152 SMs of six): a block takes several layers, whose
    rows follow one another in rounds of eight, and the last block of a sequence fewer."""
    moves = [moves[b % len(moves)] for b in range(batch)]
    c = moving(Case([m + 2 for m in moves], seed=batch, heads=heads, dim=dim, layers=layers, base=40), moves)
    got = c.check(32)
    assert got[0].tolist() == [m + 1 for m in moves]


@pytest.mark.parametrize("offset", [0, 3])
@pytest.mark.parametrize("layers", [None, 2])
def test_more_columns_than_blocks(offset, layers):
    """32768 elements of a row one by one, and 4096 chunks of it: a sequence has 64 blocks of 128 threads at most."""
    c = moving(Case([11, 2, 3], seed=5, heads=32, dim=512, layers=layers, offset=offset), [9, 0, 1])
    c.check(16)


def test_offsets_past_32_bits():
    """Rows that lie 8 GB and more behind the caches' first."""
    c = moving(Case([11, 4], seed=9, page=16, heads=8, dim=128, layers=3, base=40), [9, 2])
    pages = 1 << 17  # 4 GB a layer
    at = {p: pages - 1 - p for row in c.table for p in row if p < c.k.shape[1]}
    big = torch.empty(2, 3, pages, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
    small = c.k, c.v
    c.table = [[at.get(p, p) for p in row] for row in c.table]
    for new, old in zip(big, small):
        for p, q in at.items():
            new[:, q] = old[:, p]
    args = c.args(16)
    got = lib().nf4_tree_commit(*args, page_table=ints(c.table), k_cache=big[0], v_cache=big[1])
    c.table = [[pages - 1 - p if p < pages else p for p in row] for row in c.table]
    n, path, chosen, lens, k, v = c.want(16)
    assert [g.tolist() for g in got] == [n, path, chosen, lens]
    for new, want in zip(big, (k, v)):
        have = want.clone()
        for p, q in at.items():
            have[:, p] = new[:, q]
        assert torch.equal(c.kept(have, n).contiguous().view(torch.int16), c.kept(want, n).contiguous().view(torch.int16))
    assert lib().nf4_device_error_flags() == 0

"""nf4_kv_pages against the same steps in plain Python. Everything is whole numbers: results are equal."""
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


def lib():
    import w4a16_gemv_gb300 as nf4
    return nf4


def ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def plain(lens, counts, table, held, stack, free, page, width, first=0, depths=None, unheld=(0, 0)):
    """The documented steps on lists; table and stack are changed. unheld: tokens before and behind the sequences'."""
    need = [-(-(a + n) // page) for a, n in zip(lens, counts)]
    for b, h in enumerate(held):
        for c in range(need[b], h):
            stack[free] = table[b][c]
            free += 1
    short, fits = False, []
    for b, h in enumerate(held):
        grow = max(need[b] - h, 0)
        if need[b] > width:
            fits.append(False)
            continue
        short = short or grow > free
        fits.append(grow == 0 or not short)
        if fits[-1]:
            for c in range(h, need[b]):
                free -= 1
                table[b][c] = stack[free]
    slots, positions = [-1] * unheld[0], [0] * unheld[0]
    for b, n in enumerate(counts):
        for i in range(n):
            t = len(slots)
            key = lens[b] + i
            slots.append(table[b][key // page] * page + key % page if fits[b] else -1)
            positions.append(first + lens[b] + (i if depths is None else depths[t]))
    slots += [-1] * unheld[1]
    positions += [0] * unheld[1]
    return (slots, positions, [a + n if f else a for a, n, f in zip(lens, counts, fits)],
            [p if f else h for p, h, f in zip(need, held, fits)], [free], short, any(p > width for p in need))


class State:
    def __init__(self, rng, batch, page, longest, spare, width=None, stride=None, surplus=0.3):
        self.page = page
        self.lens = [rng.randrange(longest + 1) for _ in range(batch)]
        self.held = [max(0, -(-v // page) + rng.choice([0, 0, 1, 3]) * (rng.random() < surplus)) for v in self.lens]
        self.width = width if width is not None else max(self.held + [0]) + 40
        self.held = [min(h, self.width) for h in self.held]
        total = sum(self.held) + spare
        order = list(range(total + 5))
        rng.shuffle(order)
        at = 0
        self.table = [[-7] * self.width for _ in range(batch)]
        for b, h in enumerate(self.held):
            self.table[b][:h] = order[at:at + h]
            at += h
        self.stack = order[at:at + spare] + [-9] * (total - spare)
        self.free = spare
        stride = stride or self.width
        self.big = torch.full((batch, stride), -5, dtype=torch.int32, device="cuda")
        self.dev_table = self.big[:, :self.width]
        self.dev_table.copy_(ints(self.table).view(batch, self.width))
        self.dev = dict(lens=ints(self.lens), held=ints(self.held), free_pages=ints(self.stack), free_count=ints([self.free]))

    def check(self, counts, first=0, depths=None, in_place=False, unheld=(0, 0), single=False):
        cu = [unheld[0]]
        for n in counts:
            cu.append(cu[-1] + n)
        tokens = cu[-1] + unheld[1]
        want = plain(self.lens, counts, self.table, self.held, self.stack, self.free, self.page, self.width, first, depths,
                     unheld)
        kw = dict(new_held=self.dev["held"], new_free_count=self.dev["free_count"]) if in_place else {}
        kw.update({} if single else dict(cu_q=ints(cu), tokens=tokens))
        if depths is not None:
            kw["depths"] = ints(depths)
        got = lib().nf4_kv_pages(self.dev["lens"], self.dev_table, self.dev["held"], self.dev["free_pages"],
                                 self.dev["free_count"], self.page, first_position=first, **kw)
        names = ("slots", "positions", "new_lens", "new_held", "new_free_count")
        for name, g, w in zip(names, got, want):
            assert g.tolist() == w, name
        assert self.dev_table.tolist() == self.table and self.dev["free_pages"].tolist() == self.stack
        assert (self.big[:, self.width:] == -5).all()
        assert [int(v) for v in self.dev["lens"]] == self.lens
        if in_place:
            assert got[3] is self.dev["held"] and got[4] is self.dev["free_count"]
        assert lib().nf4_device_error_flags() == (4 if want[5] else 0) + (2 if want[6] else 0)
        self.dev.update(lens=got[2], held=got[3], free_count=got[4])
        self.lens, self.held, self.free = want[2], want[3], want[4][0]
        return got


@pytest.mark.parametrize("page", [1, 16, 24, 256])
@pytest.mark.parametrize("batch", [1, 2, 32, 255, 256, 257, 1024, 1025, 2600])
def test_one_token_each(page, batch):
    s = State(random.Random(batch + page), batch, page, 90, batch + 3, stride=None)
    s.check([1] * batch, first=11, single=True)
    s.check([1] * batch, in_place=True)


@pytest.mark.parametrize("page", [1, 5, 16, 64])
@pytest.mark.parametrize("batch,most", [(1, 3), (3, 700), (7, 40), (40, 300), (300, 25), (1500, 9), (2, 9000)])
def test_ragged_tokens(page, batch, most):
    rng = random.Random(batch * most + page)
    counts = [rng.choice([0, 1, rng.randrange(most + 1)]) for _ in range(batch)]
    s = State(rng, batch, page, 300, sum(-(-n // page) + 1 for n in counts), width=-(-(300 + most) // page) + 4, stride=None)
    s.check(counts, first=5, in_place=rng.random() < 0.5, unheld=(rng.randrange(4), rng.randrange(70)))
    # rejected tokens: shorter lengths give pages back
    s.lens = [max(0, v - rng.randrange(60)) for v in s.lens]
    s.dev["lens"] = ints(s.lens)
    s.check([0] * batch)
    s.check(counts)


def test_a_table_that_is_a_view():
    s = State(random.Random(5), 9, 16, 200, 60, stride=77)
    s.check([40, 0, 3, 100, 1, 1, 0, 20, 5])


def test_positions_by_depth():
    s = State(random.Random(6), 3, 16, 50, 30)
    s.check([4, 0, 5], first=100, depths=[0, 1, 1, 2, 0, 1, 2, 2, 3])


@pytest.mark.parametrize("batch", [5, 1300])
@pytest.mark.parametrize("spare", [0, 1, 7, 20])
def test_pages_run_out(batch, spare):
    """The first request that finds too few pages, and those after it that need some, get none; the others go on."""
    rng = random.Random(spare + batch)
    s = State(rng, batch, 8, 100, spare, surplus=0.0, width=40)
    at = s.free
    s.check([rng.choice([0, 1, 9, 30]) for _ in range(batch)])
    assert s.free <= at
    # pages that come back in the same call are there for others
    s.lens = [0 if b % 3 == 0 else v for b, v in enumerate(s.lens)]
    s.dev["lens"] = ints(s.lens)
    s.check([0 if b % 3 == 0 else 10 for b in range(batch)], in_place=True)


def test_requests_longer_than_their_row():
    s = State(random.Random(2), 4, 16, 40, 50, width=5)
    s.check([200, 3, 41, 1])


@pytest.mark.parametrize("batch", [6, 1100])
def test_a_run_of_steps_keeps_every_page_once(batch):
    rng = random.Random(batch)
    s = State(rng, batch, 4, 30, 12 * batch, width=64)
    everything = sorted(s.stack[:s.free] + [p for b in range(batch) for p in s.table[b][:s.held[b]]])
    for step in range(6):
        s.check([rng.choice([0, 1, 1, 13, 40]) if rng.random() < 0.9 else 0 for _ in range(batch)], in_place=step % 2 == 0)
        have = s.stack[:s.free] + [p for b in range(batch) for p in s.table[b][:s.held[b]]]
        assert sorted(have) == everything
        s.lens = [0 if rng.random() < 0.1 else max(0, v - rng.randrange(8)) for v in s.lens]
        s.dev["lens"] = ints(s.lens)


def test_values_out_of_range_are_clamped_and_reported():
    def run(lens=(5, 5), cu=(0, 2, 4), held=(1, 1), stack=(10, 11, 12), free=3, table=((1, -1, -1), (2, -1, -1)), tokens=4):
        t, f = ints(table), ints(stack)
        out = lib().nf4_kv_pages(ints(lens), t, ints(held), f, ints([free]), 8, cu_q=ints(cu), tokens=tokens)
        return [o.tolist() for o in out], t.tolist(), lib().nf4_device_error_flags()

    good, _, flags = run()
    assert good == [[13, 14, 21, 22], [5, 6, 5, 6], [7, 7], [1, 1], [3]] and flags == 0
    assert run(lens=(-3, 5))[2] == 2 and run(lens=(-3, 5))[0][0] == [8, 9, 21, 22]
    assert run(cu=(0, 9, 4))[2] == 2  # the second request ends before it begins
    assert run(cu=(-5, 2, 4))[0][0] == [13, 14, 21, 22]
    assert lib().nf4_device_error_flags() == 0
    assert run(cu=(0, 2, 1 << 30))[0][2] == [7, 7]
    out, _, flags = run(held=(1 << 20, 1))
    assert flags == 2 and out[3][0] == 1  # three pages, of which two go back (and do not fit there)
    assert run(held=(-4, 1))[2] == 2 and run(held=(-4, 1))[0][3] == [1, 1]
    assert run(free=99)[2] == 2 and run(free=99)[0][4] == [3]
    assert run(free=-1)[2] == 2 and run(free=-1)[0][4] == [0]
    out, _, flags = run(table=((-1, -1, -1), (2, -1, -1)))
    assert flags == 2 and out[0] == [-1, -1, 21, 22]
    out, table, flags = run(lens=(2 ** 31 - 1, 5))
    assert flags == 2 and out[0] == [-1, -1, 21, 22] and out[2] == [2 ** 31 - 1, 7]


def test_no_requests_and_no_tokens():
    none = ints([])
    out = lib().nf4_kv_pages(none, none.view(0, 3), none, ints([4, 5]), ints([2]), 16)
    assert [o.tolist() for o in out] == [[], [], [], [], [2]]
    out = lib().nf4_kv_pages(none, none.view(0, 3), none, ints([4, 5]), ints([2]), 16, cu_q=ints([0]), tokens=3)
    assert out[0].tolist() == [-1] * 3 and out[1].tolist() == [0] * 3
    assert lib().nf4_device_error_flags() == 0


@pytest.mark.parametrize("batch,most", [(20, 1), (20, 900)])
def test_recorded_and_replayed(batch, most):
    """A recorded call that works in place follows the lengths as they grow."""
    rng = random.Random(1)
    s = State(rng, batch, 16, 50, 60 * batch * max(1, most // 16), width=8 + 6 * (most // 16 + 1))
    counts = [rng.randrange(1, most + 1) for _ in range(batch)]
    cu = ints([sum(counts[:b]) for b in range(batch + 1)])
    d = s.dev
    slots, positions = torch.empty(2, sum(counts), dtype=torch.int64, device="cuda")
    new_lens = torch.empty_like(d["lens"])
    first = {k: v.clone() for k, v in d.items()}
    table = s.dev_table.clone()

    def step():
        lib().nf4_kv_pages(d["lens"], s.dev_table, d["held"], d["free_pages"], d["free_count"], 16, cu_q=cu,
                           tokens=sum(counts), slots=slots, positions=positions, new_lens=new_lens, new_held=d["held"],
                           new_free_count=d["free_count"])
        d["lens"].copy_(new_lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for k, v in first.items():
            d[k].copy_(v)
        s.dev_table.copy_(table)
        for _ in range(4):
            graph.replay()
            want = plain(s.lens, counts, s.table, s.held, s.stack, s.free, 16, s.width)
            assert slots.tolist() == want[0] and positions.tolist() == want[1]
            s.lens, s.held, s.free = want[2], want[3], want[4][0]
            assert d["held"].tolist() == s.held and d["free_count"].tolist() == [s.free] and d["lens"].tolist() == s.lens
    side.synchronize()
    assert lib().nf4_device_error_flags() == 0


def test_refusals():
    s = State(random.Random(0), 3, 16, 40, 9)
    d, t = s.dev, s.dev_table
    run = lib().nf4_kv_pages
    with pytest.raises(TypeError, match="tokens"):
        run(d["lens"], t, d["held"], d["free_pages"], d["free_count"], 16, cu_q=ints([0, 1, 2, 3]))
    with pytest.raises(TypeError, match="int32"):
        run(d["lens"].long(), t, d["held"], d["free_pages"], d["free_count"], 16)
    with pytest.raises(ValueError, match="shape"):
        run(d["lens"], t[:2], d["held"], d["free_pages"], d["free_count"], 16)
    with pytest.raises(ValueError, match="contiguous"):
        run(d["lens"], t.t().contiguous().t(), d["held"], d["free_pages"], d["free_count"], 16)
    with pytest.raises(lib().NF4Error, match="INVALID_SIZE"):
        run(d["lens"], t, d["held"], d["free_pages"], d["free_count"], 0)
    with pytest.raises(lib().NF4Error, match="INVALID_SIZE"):
        run(d["lens"], t, d["held"], d["free_pages"], d["free_count"], 16, new_lens=d["lens"])
    with pytest.raises(ValueError, match="2\\^24"):
        run(d["lens"], t, d["held"], d["free_pages"], d["free_count"], 16, cu_q=ints([0, 1, 2, 3]), tokens=1 << 40)

"""The barriers of key tiles that take turns (nf4_prefix_attn_tc.cu), as a model on the CPU.

The kernel's warps are generators that wait and arrive as they do there: a warp that copies K tiles, one that copies V tiles,
one that clears what the last V tile's copy reaches past the keys, one that issues the products, and four softmax warps for
each half of the key tiles. Copies land and products run some time after they were asked for (products in their order).
Random interleavings, some parts much slower than others in each run, look for a tile that is overwritten before it was
used or used before it is there, a barrier that is given more arrivals than its phase has, and waits that never end. The numbers of barriers and
ring tiles are read from the source. Two mistakes, planted in the model, have to be found."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_gemv_gb300", "csrc",
                      "nf4_prefix_attn_tc.cu")
BOXES = 4  # pieces in which a tile lands


def numbers():
    text = open(SOURCE).read()

    def one(pattern):
        found = re.findall(pattern, text)
        assert len(found) == 1, pattern
        return found[0]
    go, keys = int(one(r"constexpr int kGo = (\d+);")), int(one(r"constexpr int kKeys = (\d+);"))
    return go, keys, [int(x) for x in one(r"constexpr int kPairStages = DP == 128 \? (\d+) : (\d+);")]


class Fault(Exception):
    pass


def need(ok, what):
    if not ok:
        raise Fault(what)


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.bytes = self.phase = 0

    def step(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count

    def arrive(self, expect=0):
        need(self.pending > 0, "more arrivals than the phase has")
        self.bytes += expect
        self.pending -= 1
        self.step()

    def land(self):
        self.bytes -= 1
        self.step()

    def passed(self, parity):
        return self.phase & 1 != parity


def run(n, clean, stages, kgo, kkeys, seed, mistake=None):
    """One item of n key tiles; clean: the last one's copy of V reaches past the keys."""
    rng = random.Random(seed)
    go, kfirst, empty = ([Barrier(c) for _ in range(k)] for c, k in ((6, kgo), (1, kkeys), (1, stages)))
    sfull, tail = [Barrier(1), Barrier(1)], Barrier(1)
    ring = [None] * stages          # [tile number, pieces landed, cleared]
    users = [0] * stages            # products asked for that read it
    scores, weights, sums = [None, None], [[None] * 4, [None] * 4], [[], []]
    copies, products = [], []
    queued = [0, 0]                 # products into each half's O that have not run

    def load(u, bar):
        slot = u % stages
        need(users[slot] == 0, f"tile {u} is copied over one in use")
        need(ring[slot] is None, f"tile {u} is copied over one that was not used")
        ring[slot] = [u, 0, False]
        copies.extend((slot, u, bar) for _ in range(BOXES))

    def loader(kv):
        for i in range(n):
            u = 2 * i + kv
            if u >= stages:
                yield lambda: empty[u % stages].passed((u // stages - 1) & 1)
            bar = kfirst[i % kkeys] if kv == 0 else tail if clean and i + 1 == n else go[i % kgo]
            bar.arrive(BOXES)
            yield
            if kv == 1 and i + 1 < n:
                go[i % kgo].arrive()
                yield
            load(u, bar)
            yield
        if kv == (0 if mistake == "last arrival by the warp of K" else 1):
            go[(n - 1) % kgo].arrive()

    def cleaner():
        if not clean:
            return
        yield lambda: tail.passed(0)
        tile = ring[(2 * n - 1) % stages]
        need(tile is not None and tile[:2] == [2 * n - 1, BOXES], "the last tile is cleared before it is there")
        tile[2] = True
        yield
        go[(n - 1) % kgo].arrive()

    def product(kind, i):
        slot = (2 * i + (kind == "o")) % stages
        users[slot] += 1
        if kind == "o":
            queued[i & 1] += 1
        products.append((kind, i, slot))

    def commit(bar):
        products.append(("commit", bar, None))

    def issuer():
        def s(i):
            yield lambda: kfirst[i % kkeys].passed(i // kkeys & 1)
            product("s", i)
            commit(sfull[i & 1])
            commit(empty[2 * i % stages])
            yield
        yield from s(0)
        yield from s(1)
        for i in range(n):
            if mistake != "no wait for the softmax":
                yield lambda: go[i % kgo].passed(i // kgo & 1)
            product("o", i)
            commit(empty[(2 * i + 1) % stages])
            yield
            if i + 2 < n:
                yield from s(i + 2)
            else:
                commit(sfull[i & 1])
                yield
        yield lambda: empty[(2 * n - 1) % stages].passed((2 * n - 1) // stages & 1)

    def softmax(half, warp):
        for i in range(half, n, 2):
            yield lambda: sfull[half].passed(i >> 1 & 1)
            need(scores[half] == i, f"scores of tile {i} are not there")
            need(queued[half] == 0, f"O of tile {i} is not at rest")
            yield
            need(scores[half] == i, f"scores of tile {i} are overwritten")
            weights[half][warp] = i
            yield
            go[i % kgo].arrive()
        yield lambda: sfull[half].passed(((n + 1) >> 1 if half == 0 else n >> 1) & 1)
        need(sums[half] == list(range(half, n, 2)), "products are missing at the end")

    def tensor_cores():
        kind, i, slot = products.pop(0)
        if kind == "commit":
            return i.arrive()
        tile = ring[slot]
        need(tile is not None and tile[:2] == [2 * i + (kind == "o"), BOXES], f"a product reads a tile that is not there: {kind}{i}")
        if kind == "s":
            need(all(w == (i - 2 if i > 1 else None) for w in weights[i & 1]), "scores are written over ones in use")
            scores[i & 1] = i
        else:
            need(tile[2] or not (clean and i + 1 == n), "the last tile is not cleared")
            need(all(w == i for w in weights[i & 1]), f"weights of tile {i} are not there")
            sums[i & 1].append(i)
            queued[i & 1] -= 1
        users[slot] -= 1
        ring[slot] = None

    def copy():
        slot, u, bar = copies.pop(rng.randrange(len(copies)))
        need(ring[slot] is not None and ring[slot][0] == u, "a copy lands in a tile that was given away")
        ring[slot][1] += 1
        bar.land()

    parts = {"k": loader(0), "v": loader(1), "clean": cleaner(), "issue": issuer(),
             **{f"softmax {h} {w}": softmax(h, w) for h in (0, 1) for w in range(4)}}
    waits = {name: None for name in parts}
    speed = {name: rng.choice((1, 1, 5, 40)) for name in [*parts, "tensor", "copy"]}
    while parts or products or copies:
        ready = [name for name in parts if waits[name] is None or waits[name]()]
        ready += ["tensor"] * bool(products) + ["copy"] * bool(copies)
        need(ready, f"waits that never end: {sorted(parts)}")
        name = rng.choices(ready, [speed[r] for r in ready])[0]
        if name == "tensor":
            tensor_cores()
        elif name == "copy":
            copy()
        else:
            try:
                waits[name] = next(parts[name])
            except StopIteration:
                del parts[name], waits[name]


@pytest.mark.parametrize("stages", [0, 1], ids=["128 elements", "64 elements"])
@pytest.mark.parametrize("clean", [False, True], ids=["whole", "cleared"])
def test_key_tiles_in_turns(stages, clean):
    go, keys, rings = numbers()
    for n in range(2, 21):
        for seed in range(30 if n < 10 else 8):
            run(n, clean, rings[stages], go, keys, f"{n} {seed}")


@pytest.mark.parametrize("mistake", ["last arrival by the warp of K", "no wait for the softmax"])
def test_the_model_finds_mistakes(mistake):
    go, keys, rings = numbers()
    found = 0
    for seed in range(400):
        try:
            run(9, False, rings[seed % 2], go, keys, seed, mistake)
        except Fault:
            found += 1
    assert found >= 20, found

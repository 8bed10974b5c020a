"""nf4_prefix_attention for batches of many sequences: every tile finds its own, and in the same time however many there are.
Tolerances are those of test_gpu_prefix_attention.py."""
import pytest
import torch

from test_gpu_prefix_attention import Call, lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hk", [(6, 2), (1, 1), (40, 2)])
@pytest.mark.parametrize("batch", [31, 32, 33, 64, 65, 1024, 1500])
def test_many_sequences(hq, hk, batch):
    """One token each by division, by the search, and with sequences without tokens among them."""
    lens = [(b * 37) % 90 for b in range(batch)]
    c = Call(hq, hk, 64, 70, lens, [1] * batch, seed=batch)
    first = c.run()
    c.check(first, "search")
    again = c.run(cu_q=None)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    counts = [(0, 1, 0, 3, 1, 0, 0, 17)[(b * 5 + b // 8) % 8] for b in range(batch)]
    c = Call(hq, hk, 64, 70, lens, counts, seed=batch + 1)
    c.check(c.run(), "ragged")


@pytest.mark.parametrize("most", [60, 150])
@pytest.mark.parametrize("batch", [33, 70, 1100])
@pytest.mark.parametrize("prefix", [0, 300])
def test_many_sequences_of_many_rows(prefix, batch, most):
    """Tiles of 64 and of 256 rows."""
    counts = [most - (b * 31) % (most // 2) for b in range(batch)]
    counts[batch // 2] = 0
    counts[-1] = 2 * most
    c = Call(1, 1, 64, prefix, [n + b % 50 for b, n in enumerate(counts)], counts, seed=batch + most)
    c.check(c.run())


def test_cu_q_is_checked_wherever_it_is_wrong():
    """One falling entry of a large batch, wherever it stands, sets the flag."""
    nf4 = lib()
    batch = 700
    c = Call(2, 1, 64, 20, [5] * batch, [1] * batch, seed=3)
    for at in (1, 33, 350, 640, 699):
        cu = c.cu_q.clone()
        cu[at] += 2
        c.run(cu_q=cu)
        torch.cuda.synchronize()
        assert nf4.nf4_device_error_flags() == 2, at
    few = Call(2, 1, 64, 20, [5] * batch, [0] * (batch - 2) + [1, 1], seed=3)  # few tiles, many sequences
    few.check(few.run())
    cu = few.cu_q.clone()
    cu[300] = 1
    few.run(cu_q=cu)
    torch.cuda.synchronize()
    assert nf4.nf4_device_error_flags() == 2


@pytest.mark.parametrize("cu", [False, True], ids=["one each", "cu_q"])
def test_time_grows_with_the_batch_and_not_with_its_square(cu):
    """200 own keys of two heads each. A scan of the batch for every tile took 4 times as long per sequence at 16384 as at 2048;
    2 leaves room for the noise of a shared machine."""
    page, keys, nf4 = 64, 200, lib()
    cache = torch.randn(64, page, 2, 64, device="cuda").bfloat16()
    none = torch.empty(0, dtype=torch.int32, device="cuda")

    def time(batch):
        pages = torch.randint(0, 64, (batch, 4), device="cuda", dtype=torch.int32)
        lens = torch.full((batch,), keys, device="cuda", dtype=torch.int32)
        q = torch.randn(batch, 2, 64, device="cuda").bfloat16()
        cu_q = torch.arange(batch + 1, device="cuda", dtype=torch.int32) if cu else None
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            nf4.nf4_prefix_attention(q, cache, cache, none, 0, pages, lens, cu_q=cu_q)
            a.record()
            for _ in range(5):
                nf4.nf4_prefix_attention(q, cache, cache, none, 0, pages, lens, cu_q=cu_q)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best / batch

    assert time(16384) <= 2 * time(2048)

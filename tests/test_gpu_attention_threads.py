"""The compiled entry points beside other Python threads."""
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["rotation", "append", "attention"])
def test_other_threads_run_while_a_launch_waits(name):
    """Launches behind a kernel of about half a second, more of them than a stream's queue holds: the calls wait for room, and
    a thread that looks at the clock is not kept waiting with them (held up, it would see a gap of that half second)."""
    import w4a16_gemv_gb300 as nf4
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    table = nf4.nf4_rope_table(4, 64)
    pages = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    call = {"rotation": lambda: nf4.nf4_qk_norm_rope(x, x, pos, table, q_out=a, k_out=b),
            "append": lambda: nf4.nf4_kv_append(cache, cache, pos, x, x, pos, table, q=x, q_out=a),
            "attention": lambda: nf4.nf4_prefix_attention(x, cache, cache, pages[0], 0, pages, lens, out=a)}[name]
    call()
    torch.cuda.synchronize()
    gaps, done = [], threading.Event()

    def watch():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    thread = threading.Thread(target=watch)
    torch.cuda._sleep(1_000_000_000)  # cycles
    start = time.perf_counter()
    thread.start()
    for _ in range(3000):
        call()
    waited = time.perf_counter() - start
    done.set()
    thread.join()
    torch.cuda.synchronize()
    assert waited > 0.25, "the queue never filled"
    assert max(gaps) < 0.15, max(gaps)

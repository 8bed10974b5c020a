"""nf4_device_error_flags: every kernel's bits at once, and in the time of a few small copies."""
import time

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_flags_of_several_kernels_are_read_and_cleared_together():
    import w4a16_gemv_gb300 as nf4
    x = torch.randn(2, 2, 64, device="cuda").bfloat16()
    pages = torch.randn(2, 16, 2, 64, device="cuda").bfloat16()
    table = nf4.nf4_rope_table(10, 64)
    ints = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0], [[1], [1]], [3, 99])]
    good, bad = (torch.tensor(v, device="cuda") for v in ([3, 4], [3, 10]))

    def rope(pos):
        nf4.nf4_qk_norm_rope(x, x, pos, table)

    def attend(lens):
        nf4.nf4_prefix_attention(x, pages, pages, ints[0], 16, ints[1], lens)

    assert nf4.nf4_device_error_flags() == 0
    for calls, want in (((lambda: rope(bad),), 2), ((lambda: attend(ints[2]),), 2),
                        ((lambda: rope(bad), lambda: attend(ints[2])), 2),
                        ((lambda: rope(good), lambda: attend(ints[2].clamp(max=16))), 0)):
        for call in calls:
            call()
        assert nf4.nf4_device_error_flags() == want
        assert nf4.nf4_device_error_flags() == 0


def test_time_of_a_look_at_the_flags():
    """At most three small reads from the device. With a read and a write of their own for each of four words it was six."""
    import w4a16_gemv_gb300 as nf4
    word = torch.zeros(1, device="cuda")

    def best(call):
        times = []
        for _ in range(20):
            t = time.perf_counter()
            for _ in range(20):
                call()
            times.append(time.perf_counter() - t)
        return min(times)

    assert best(nf4.nf4_device_error_flags) <= 3 * best(word.item)

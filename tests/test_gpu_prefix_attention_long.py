"""nf4_prefix_attention over ranges of a million keys, on caches of two pages that the page tables repeat."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def lib():
    import w4a16_gemv_gb300 as nf4
    return nf4


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("n", [1 << 17, 1 << 20])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("shared", [True, False], ids=["tcgen05", "mma.sync"])
def test_small_weights_beside_a_large_one(shared, dt, n):
    """One key of score 26 ln 2 and n - 1 of score 0, whose weights are w = 2^-26 of the first one's (in binary16 below
    half the smallest number) and together t = (n - 1) w. Column 0 of v is 0 at that key and 1 elsewhere, so that the output
    is t / (1 + t), all of it of small weights; column 1 is 1 throughout.

    What is added to a sum that holds the first key may be lost, w at a time: a range, of 2^17 keys at most, loses up to
    2^17 w = 2^-9 = a in l and in column 1. Column 0 holds no large weight and is exact (sums of powers of two within 24
    bits). So |out0 - t / (1 + t)| <= t (a + u) + 2^-25, |out1 - 1| <= a + u, |lse - exact| <= a + 1e-5."""
    page = 1 << 16
    k = torch.zeros(2, page, 1, 8, dtype=dt, device="cuda")
    k[0, 5, 0, 0] = 26
    v = torch.ones_like(k)
    v[0, 5, 0, 0] = 0
    table = ints(0, *[1] * (n // page - 1))
    heads, tokens = (64, 608) if shared else (1, 1216)  # a row tile on every SM: as few ranges as there may be
    q = torch.zeros(tokens, heads, 8, dtype=dt, device="cuda")
    q[..., 0] = 1
    if shared:
        args, cu = (table, n, torch.empty(1, 0, dtype=torch.int32, device="cuda"), ints(0)), ints(0, tokens)
    else:
        args, cu = (ints(), 0, table.expand(tokens, -1), ints(*[n] * tokens)), None
    out, lse = lib().nf4_prefix_attention(q, k, v, *args, cu_q=cu, scale=math.log(2.0), return_lse=True)
    t, a, u = (n - 1) * 2.0 ** -26, 2.0 ** -9, {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dt]
    out, lse = out.double(), lse.double()
    assert float((out[..., 0] - t / (1 + t)).abs().max()) <= t * (a + u) + 2.0 ** -25
    assert float((out[..., 1:] - 1).abs().max()) <= a + u
    assert float((lse - 26 * math.log(2.0) - math.log1p(t)).abs().max()) <= a + 1e-5
    assert lib().nf4_device_error_flags() == 0

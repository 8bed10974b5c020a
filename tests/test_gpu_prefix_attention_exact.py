"""nf4_prefix_attention over long ranges with inputs whose sums are exact, so that a single key lost, repeated or read from
another page shows.

Key j of a sequence (the shared ones first) is a unit vector along column (j / 16) % dim, its value one along column
(5 (j / 8) + 1) % dim. Query head h is 4 along column COLUMNS[h % 4], and the scale ln 2: a key's score is 4 ln 2 where its column
is the head's and 0 elsewhere, its weight 16 or 1 times a power of two. Sums of fewer than 2^17 such weights are exact in
binary32, in any order and however the keys are cut. What is left, relative: exp2 (2^-22), the logarithm and its sum (8 e of lse),
1 / l and the product (2^-20 with the former), and the result's own rounding u (in binary16 also 2^-25).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E = 2.0 ** -24
COLUMNS = (0, 3, -2, -1)


def column(j, dim):
    return (j // 16) % dim, (5 * (j // 8) + 1) % dim


def expected(n, dim):
    """lse [4, n + 1] and out [4, n + 1, dim] of rows that see the first 0 .. n keys, in binary64."""
    j = torch.arange(n, device="cuda")
    kc, vc = column(j, dim)
    mine = torch.tensor([c % dim for c in COLUMNS], device="cuda")
    w = torch.where(kc[None] == mine[:, None], 16.0, 1.0).double()
    out = torch.zeros(4, n + 1, dim, dtype=torch.float64, device="cuda")
    out[:, 1:][:, j, vc] = w
    out = out.cumsum(1)
    total = out.sum(-1)
    return total.log(), out / total.clamp(min=1)[..., None]


def run(hq, hk, dim, prefix, lens, counts, page, dt, shared_rows=False):
    """`shared_rows`: the sequences have the same own pages."""
    need = [-(-n // page) for n in (lens[:1] if shared_rows else lens)]
    shared = -(-prefix // page)
    order = torch.randperm(shared + sum(need) + 2, device="cuda").int()
    k, v = (torch.full((len(order), page, hk, dim), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    unit = torch.eye(dim, dtype=dt, device="cuda")

    def fill(table, first, n):
        j = torch.arange(n, device="cuda")
        p = table[j // page].long()
        kc, vc = column(first + j, dim)
        k[p, j % page] = unit[kc][:, None]
        v[p, j % page] = unit[vc][:, None]

    prefix_pages = order[:shared].contiguous()
    fill(prefix_pages, 0, prefix)
    suffix_pages = torch.full((len(need), max(need)), -1, dtype=torch.int32, device="cuda")
    at = shared
    for b, n in enumerate(need):
        suffix_pages[b, :n] = order[at:at + n]
        fill(suffix_pages[b], prefix, lens[b])
        at += n
    if shared_rows:
        suffix_pages = suffix_pages.expand(len(lens), -1)
    q = torch.zeros(sum(counts), hq, dim, dtype=dt, device="cuda")
    for h in range(hq):
        q[:, h, COLUMNS[h % 4]] = 4
    cu = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    import w4a16_gemv_gb300 as nf4
    out, lse = nf4.nf4_prefix_attention(q, k, v, prefix_pages, prefix, suffix_pages,
                                        torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_q=cu, scale=math.log(2.0),
                                        return_lse=True)
    want_lse, want = expected(prefix + max(lens), dim)
    # keys that each token sees, and its heads' rows of the tables
    sees = torch.cat([prefix + max(n, 0) - c + 1 + torch.arange(c) for n, c in zip(lens, counts)]).cuda()
    head = torch.arange(hq, device="cuda") % 4
    want_lse, want = want_lse[head[None], sees[:, None]], want[head[None], sees[:, None]]
    tol = 2.0 ** -22 + 8 * E * want_lse.abs()
    # eight keys of weight 1 more or less would be seen
    assert float((8 / want_lse.exp()).min()) > 4 * float(tol.max())
    err = (lse.double() - want_lse).abs()
    assert (err <= tol).all(), f"lse: {float((err / tol).max()):.2f} x"
    tol = (U[dt] + 2.0 ** -20) * want + (2.0 ** -25 if dt == torch.float16 else 0.0)
    err = (out.double() - want).abs()
    assert (err <= tol).all(), f"out: {float((err / tol.clamp(min=1e-30)).max()):.2f} x"
    assert nf4.nf4_device_error_flags() == 0


DT = pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
PAGES = pytest.mark.parametrize("page", [12, 16, 24, 64, 136])  # 12: without tensor copies


@DT
@PAGES
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("prefix", [70001, 16384, 4113])
def test_shared_keys_in_many_ranges(dt, page, dim, prefix):
    run(12, 2, dim, prefix, [17, 200, 33], [1, 2, 1], page, dt)


@DT
@PAGES
@pytest.mark.parametrize("dim", [64, 128])
def test_shared_keys_in_few_ranges(dt, page, dim):
    """A row tile and more on every SM: one range, and with half of them two."""
    for tokens in (640, 320):
        run(64, 1, dim, 30001, [tokens + 40], [tokens], page, dt)


@DT
@PAGES
@pytest.mark.parametrize("dim", [64, 128])
def test_own_keys_of_few_rows(dt, page, dim):
    run(4, 2, dim, 0, [70003, 20000, 9], [1, 1, 1], page, dt)
    run(4, 4, dim, 20, [3001] * 400, [1] * 400, page, dt, shared_rows=True)


@DT
@PAGES
@pytest.mark.parametrize("dim", [64, 128])
def test_own_keys_of_many_rows(dt, page, dim):
    run(8, 1, dim, 0, [40011, 9000], [250, 60], page, dt)
    run(8, 1, dim, 5000, [2500, 1200], [1000, 900], page, dt)

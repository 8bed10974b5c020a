"""nf4_rope_table, nf4_qk_norm_rope and nf4_kv_append against their formulas in binary64.

Tolerances. With u the unit roundoff of the dtype (2^-8, 2^-11, 2^-24) and e = 2^-24: the sum of
squares of D terms is within D e of exact, relatively; the norm's factor takes half of that, and
the products, the table and the rotation a few e more, each relative to |a| + |b| of the pair. So
|y - y_exact| <= u |y_exact| + (D / 2 + 16) e (|a| + |b|) + tiny, with tiny half the smallest
subnormal of the dtype (2^-134, 2^-25, 2^-150; in binary32 also the flushed part of rsqrt: 2^-126).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -126}
E = 2.0 ** -24


def lib():
    import w4a16_gemv_gb300 as nf4
    return nf4


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def frequencies(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def angles(positions, freqs):
    """cos and sin in binary64 of integer positions: [n, pairs]."""
    a = positions.double()[:, None] * torch.tensor(freqs, dtype=torch.float64, device=positions.device)
    return torch.cos(a), torch.sin(a)


def expected(x, weight, cos, sin, interleaved, eps):
    """(values, |a| + |b| of each element's pair) in binary64 for rows x [tokens, heads, dim]."""
    u = x.double()
    if weight is not None:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + eps) * weight.double()
    y, mag = u.clone(), u.abs()
    half = cos.shape[1]
    if half:
        i = torch.arange(half, device=x.device)
        p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b, c, s = u[..., p], u[..., r], cos[:, None], sin[:, None]
        y[..., p], y[..., r] = a * c - b * s, b * c + a * s
        mag[..., p] = mag[..., r] = a.abs() + b.abs()
    return y, mag


def check(got, want, what):
    y, mag = want
    dt, dim = got.dtype, got.shape[-1]
    tol = U[dt] * y.abs() + (dim / 2 + 16) * E * mag + TINY[dt]
    err = (got.double() - y).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst {float((err / tol).max()):.2f} x"


def inputs(tokens, hq, hk, dim, dt, seed, max_pos):
    g = gen(seed)
    qkv = torch.randn(tokens, hq + 2 * hk, dim, device="cuda", generator=g).to(dt)
    pos = torch.randint(0, max_pos, (tokens,), device="cuda", generator=g)
    w = [(1 + 0.3 * torch.randn(dim, device="cuda", generator=g)).to(dt) for _ in range(2)]
    return qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:], pos, w[0], w[1]


# ------------------------------------------------------------------------------------ the table

@pytest.mark.parametrize("rot,base,n", [(128, 10000.0, 4097), (2, 10000.0, 300), (96, 500000.0, 1000), (512, 1e6, 33)])
def test_table_plain(rot, base, n):
    t = lib().nf4_rope_table(n, rot, base=base)
    cos, sin = angles(torch.arange(n, device="cuda"), frequencies(rot, base))
    # sincosf within 2 units in the last place of a value below 1, the first-order term and one rounding
    assert (t[..., 0].double() - cos).abs().max() <= 3e-7 and (t[..., 1].double() - sin).abs().max() <= 3e-7


def test_table_far_rows():
    """Row 2^24 - 1 of a long table is as exact as the first: the angle is reduced in binary64."""
    n = 1 << 24
    t = lib().nf4_rope_table(n, 4, base=100.0)
    p = torch.tensor([0, 1, n // 3, n - 2, n - 1], device="cuda")
    cos, sin = angles(p, frequencies(4, 100.0))
    assert (t[p, :, 0].double() - cos).abs().max() <= 3e-7 and (t[p, :, 1].double() - sin).abs().max() <= 3e-7


@pytest.mark.parametrize("scaling", ["linear", "bands", "ramp"])
@pytest.mark.parametrize("rot", [64, 128])
def test_table_scalings(scaling, rot):
    factor, low, high, original, mag, base = 8.0, 1.0, 4.0, 2048.0, 1.2, 10000.0
    if scaling == "ramp":
        high = 32.0
    freqs = []
    for i, f in enumerate(frequencies(rot, base)):
        if scaling == "linear":
            g = f / factor
        elif scaling == "bands":
            wave = 2 * math.pi / f
            if wave < original / high:
                g = f
            elif wave > original / low:
                g = f / factor
            else:
                s = (original / wave - low) / (high - low)
                g = (1 - s) * f / factor + s * f
        else:
            def dim_of(turns):
                return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
            lo, hi = max(math.floor(dim_of(high)), 0), min(math.ceil(dim_of(low)), rot - 1)
            s = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            g = (1 - s) * f + s * f / factor
        freqs.append(g)
    # several distinct regions are present
    ratios = {round(g / f, 6) for g, f in zip(freqs, frequencies(rot, base))}
    assert len(ratios) == 1 if scaling == "linear" else {1.0, 0.125} < ratios
    t = lib().nf4_rope_table(3000, rot, base=base, scaling=scaling, factor=factor, low=low, high=high,
                             original_positions=original, magnitude=mag)
    cos, sin = angles(torch.arange(3000, device="cuda"), freqs)
    assert (t[..., 0].double() - mag * cos).abs().max() <= 3e-7 * mag
    assert (t[..., 1].double() - mag * sin).abs().max() <= 3e-7 * mag


# ------------------------------------------------------------------------- the norm and rotation

@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("norm", [False, True], ids=["plain", "norm"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", [
    (1, 12, 2, 128, 128), (37, 12, 2, 128, 64), (5, 3, 1, 64, 16), (130, 32, 32, 128, 128), (19, 10, 2, 80, 80),
    (7, 6, 6, 96, 32), (3, 5, 3, 20, 20), (4, 1, 1, 256, 128), (2, 3, 1, 512, 512), (6, 2, 1, 34, 6), (9, 1, 1, 1, 0),
    (5, 4, 2, 64, 0), (3, 2, 2, 40, 8), (2, 1, 1, 129, 128)])
def test_norm_and_rotation(dt, interleaved, norm, tokens, hq, hk, dim, rot):
    q, k, _, pos, qw, kw = inputs(tokens, hq, hk, dim, dt, tokens * dim + rot, 5000)
    t = lib().nf4_rope_table(5000, rot) if rot else torch.empty(5000, 0, 2, device="cuda")
    qo, ko = lib().nf4_qk_norm_rope(q, k, pos, t, q_weight=qw if norm else None, k_weight=kw if norm else None,
                                    eps=1e-5, interleaved=interleaved)
    cos, sin = angles(pos, frequencies(rot))
    check(qo, expected(q, qw if norm else None, cos, sin, interleaved, 1e-5), "q")
    check(ko, expected(k, kw if norm else None, cos, sin, interleaved, 1e-5), "k")
    assert lib().nf4_device_error_flags() == 0


@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 32), (36, 20)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_one_weight_and_odd_strides(dim, rot, interleaved):
    """Outputs may be the inputs; a norm of one of the two; rows at any element offset and stride."""
    dt = torch.bfloat16
    g = gen(5)
    t = lib().nf4_rope_table(400, rot)
    pos = torch.randint(0, 400, (23,), device="cuda", generator=g)
    kw = (1 + 0.2 * torch.randn(dim, device="cuda", generator=g)).to(dt)
    for shift in (0, 1):
        buf = torch.randn(23 * (9 * dim + 5) + 8, device="cuda", generator=g).to(dt)
        q = buf[shift:].as_strided((23, 5, dim), (9 * dim + 5 * shift, dim + shift, 1))
        k = buf.as_strided((23, 2, dim), (9 * dim + 5 * shift, dim + shift, 1), 6 * dim + 2 * shift)
        before = buf.clone()
        cos, sin = angles(pos, frequencies(rot))
        want_q, want_k = expected(q, None, cos, sin, interleaved, 1e-6), expected(k, kw, cos, sin, interleaved, 1e-6)
        apart = lib().nf4_qk_norm_rope(q, k, pos, t, k_weight=kw, interleaved=interleaved)
        assert torch.equal(buf, before)
        out = lib().nf4_qk_norm_rope(q, k, pos, t, k_weight=kw, interleaved=interleaved, q_out=q, k_out=k)
        assert out[0] is q and torch.equal(q, apart[0]) and torch.equal(k, apart[1])
        check(q, want_q, "q")
        check(k, want_k, "k")
        touched = torch.zeros_like(buf, dtype=torch.bool)
        touched[shift:].as_strided(q.shape, q.stride()).fill_(True)
        touched.as_strided(k.shape, k.stride(), k.storage_offset()).fill_(True)
        assert torch.equal(buf[~touched], before[~touched])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,shift", [
    (70, 10, 2, 80, 40, 0), (11, 3, 1, 8, 8, 0), (6, 5, 3, 24, 8, 0), (9, 4, 4, 256, 40, 0), (3, 2, 1, 264, 24, 0),
    (13, 6, 2, 128, 128, 4), (13, 6, 2, 128, 64, 2), (900, 7, 3, 80, 40, 4), (3100, 2, 1, 40, 24, 0)])
def test_rows_that_fit_smaller_chunks(dt, interleaved, tokens, hq, hk, dim, rot, shift):
    """Rotated parts, offsets and strides that are multiples of 8 bytes only (and, shift 2, of 4 or 8)."""
    _, _, _, pos, qw, kw = inputs(tokens, hq, hk, dim, dt, dim + rot, 700)
    ts, hs = (hq + hk + 1) * (dim + shift) + shift, dim + shift
    buf = torch.randn(tokens * ts + 2 * shift, device="cuda", generator=gen(rot)).to(dt)
    q = buf.as_strided((tokens, hq, dim), (ts, hs, 1), shift)
    k = buf.as_strided((tokens, hk, dim), (ts, hs, 1), shift + hq * hs)
    before = buf.clone()
    t = lib().nf4_rope_table(700, rot)
    cos, sin = angles(pos, frequencies(rot))
    for wq, wk in ((qw, kw), (None, kw)):
        qo, ko = lib().nf4_qk_norm_rope(q, k, pos, t, q_weight=wq, k_weight=wk, interleaved=interleaved)
        check(qo, expected(q, wq, cos, sin, interleaved, 1e-6), "q")
        check(ko, expected(k, wk, cos, sin, interleaved, 1e-6), "k")
    want = qo.clone(), ko.clone()
    lib().nf4_qk_norm_rope(q, k, pos, t, k_weight=kw, interleaved=interleaved, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    touched = torch.zeros_like(buf, dtype=torch.bool)
    for x in (q, k):
        touched.as_strided(x.shape, x.stride(), x.storage_offset()).fill_(True)
    assert torch.equal(buf[~touched], before[~touched])


@pytest.mark.parametrize("shift", [0, 4, 1], ids=["16-byte", "8-byte", "2-byte"])
@pytest.mark.parametrize("dim,rot", [(80, 40), (128, 64), (24, 24)])
def test_append_at_smaller_alignments(dim, rot, shift):
    """Caches whose slots are a multiple of 16, 8 or 2 bytes apart."""
    nf4, dt, tokens, hk, page = lib(), torch.bfloat16, 50, 3, 16
    _, k, v, pos, _, kw = inputs(tokens, 1, hk, dim, dt, dim, 900)
    t = nf4.nf4_rope_table(900, rot)
    base = torch.randn(2, 6, page, hk, dim + shift, device="cuda", generator=gen(2)).to(dt)
    before = base.clone()
    kc, vc = base[0, ..., shift:], base[1, ..., :dim]
    slots = torch.randperm(6 * page, device="cuda", generator=gen(4))[:tokens].contiguous()
    nf4.nf4_kv_append(kc, vc, slots, k, v, pos, t, k_weight=kw)
    cos, sin = angles(pos, frequencies(rot))
    check(kc[slots // page, slots % page], expected(k, kw, cos, sin, False, 1e-6), "k")
    assert torch.equal(vc[slots // page, slots % page], v)
    other = torch.ones(6, page, dtype=torch.bool, device="cuda")
    other[slots // page, slots % page] = False
    for i in range(2):
        assert torch.equal(base[i][other], before[i][other])
    if shift:
        assert torch.equal(base[0, ..., :shift], before[0, ..., :shift])
        assert torch.equal(base[1, ..., dim:], before[1, ..., dim:])


def test_heads_far_apart():
    """A head stride whose offsets pass 32 bits, of the inputs and of the outputs."""
    dt, step = torch.bfloat16, (1 << 30) + 16
    g = gen(3)
    buf = torch.empty(2 * step + 3 * 128, dtype=dt, device="cuda")
    far = buf.as_strided((3, 3, 128), (128, step, 1))
    near = torch.randn(3, 3, 128, device="cuda", generator=g).to(dt)
    far.copy_(near)
    pos = torch.tensor([5, 0, 29], device="cuda")
    t = lib().nf4_rope_table(30, 128)
    w = (1 + 0.2 * torch.randn(128, device="cuda", generator=g)).to(dt)
    cos, sin = angles(pos, frequencies(128))
    a, b = lib().nf4_qk_norm_rope(far, near, pos, t, q_weight=w, k_weight=w)
    check(a, expected(near, w, cos, sin, False, 1e-6), "q")
    out = lib().nf4_qk_norm_rope(near, near, pos, t, q_weight=w, k_weight=w, q_out=far)
    check(out[0], expected(near, w, cos, sin, False, 1e-6), "q")
    assert torch.equal(out[1], b)


def test_extreme_rows():
    """Rows of zeros, of the largest and of subnormal values, and rows with infinities and NaN (which stay in
    their row)."""
    for dt in (torch.bfloat16, torch.float16):
        x = torch.randn(6, 4, 128, device="cuda", generator=gen(9)).to(dt)
        x[0] = 0
        x[1] = 200.0
        x[2] = torch.finfo(dt).tiny
        pos = torch.arange(6, device="cuda")
        t = lib().nf4_rope_table(6, 128)
        w = torch.ones(128, dtype=dt, device="cuda")
        cos, sin = angles(pos, frequencies(128))
        q, _ = lib().nf4_qk_norm_rope(x, x, pos, t, q_weight=w, eps=1e-6)
        check(q, expected(x, w, cos, sin, False, 1e-6), "q")
        assert torch.equal(q[0], torch.zeros_like(q[0]))
        clean = q.clone()
        x[3, 1, 5] = float("inf")
        x[4, 2, 7] = float("nan")
        q, k = lib().nf4_qk_norm_rope(x, x, pos, t, q_weight=w, eps=1e-6)
        keep = torch.ones(6, 4, dtype=torch.bool, device="cuda")
        keep[3, 1] = keep[4, 2] = False
        assert torch.equal(q[keep], clean[keep]) and q[4, 2].isnan().all() and q[3, 1].isnan().any()
        assert int(k[4, 2].isnan().sum()) == 2 and not k[keep].isnan().any()


@pytest.mark.parametrize("dim", [128, 36])
def test_position_out_of_range(dim):
    """The token's rows become NaN and the flag is set; the other tokens are as without it."""
    dt = torch.bfloat16
    q, k, _, pos, qw, _ = inputs(9, 4, 2, dim, dt, 3, 50)
    t = lib().nf4_rope_table(50, 16)
    good = lib().nf4_qk_norm_rope(q, k, pos, t, q_weight=qw)
    for bad in (-1, 50, 1 << 40):
        p = pos.clone()
        p[4] = bad
        out = lib().nf4_qk_norm_rope(q, k, p, t, q_weight=qw)
        assert lib().nf4_device_error_flags() == 2 and lib().nf4_device_error_flags() == 0
        others = [i for i in range(9) if i != 4]
        for o, w in zip(out, good):
            assert o[4].isnan().all() and torch.equal(o[others], w[others])


def test_many_tokens_and_a_side_stream():
    q, k, _, pos, qw, kw = inputs(20000, 32, 8, 128, torch.bfloat16, 8, 30000)
    t = lib().nf4_rope_table(30000, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    lib().nf4_qk_norm_rope(q, k, pos, t, q_weight=qw, k_weight=kw, q_out=qo, k_out=ko, stream=side)
    side.synchronize()
    cos, sin = angles(pos, frequencies(128))
    check(qo, expected(q, qw, cos, sin, False, 1e-6), "q")
    check(ko, expected(k, kw, cos, sin, False, 1e-6), "k")


def test_refusals_of_the_binding():
    nf4 = lib()
    q, k, v, pos, qw, _ = inputs(3, 4, 2, 64, torch.bfloat16, 1, 10)
    t = nf4.nf4_rope_table(10, 64)
    with pytest.raises(ValueError):
        nf4.nf4_qk_norm_rope(q[:2], k, pos, t)
    with pytest.raises(TypeError):
        nf4.nf4_qk_norm_rope(q.float(), k, pos, t)
    with pytest.raises(TypeError):
        nf4.nf4_qk_norm_rope(q, k, pos.int(), t)
    with pytest.raises(ValueError):
        nf4.nf4_qk_norm_rope(q, k, pos, t[:, :, 0])
    with pytest.raises(ValueError):
        nf4.nf4_qk_norm_rope(q, k, pos, t, q_weight=qw[:32])
    with pytest.raises(ValueError):
        nf4.nf4_qk_norm_rope(q.cpu(), k.cpu(), pos.cpu(), t.cpu())
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_qk_norm_rope(q, k, pos, nf4.nf4_rope_table(10, 66))  # rotates more than the head
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_rope_table(10, 63 + 512)
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, device="cuda")
    with pytest.raises(ValueError):
        nf4.nf4_kv_append(cache, cache[:, :8], slots, k, v, pos, t)
    with pytest.raises(TypeError):
        nf4.nf4_kv_append(cache, cache, slots.int(), k, v, pos, t)
    with pytest.raises(TypeError):
        nf4.nf4_kv_append(cache.half(), cache.half(), slots, k, v, pos, t)
    with pytest.raises(ValueError):
        nf4.nf4_kv_append(cache, cache, slots, k, v[:, :1], pos, t)


# ---------------------------------------------------------------------------------- the append

@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("heads_first", [False, True], ids=["slots-heads", "heads-slots"])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot,page,interleaved,norm", [
    (1, 12, 2, 128, 128, 16, False, False), (64, 12, 2, 128, 128, 16, False, True), (33, 0, 4, 64, 32, 24, True, False),
    (257, 32, 32, 128, 128, 64, False, True), (17, 6, 6, 96, 96, 1, True, True), (40, 5, 1, 30, 30, 7, False, True),
    (8, 4, 2, 80, 16, 128, False, False), (5, 2, 1, 72, 24, 3, False, False)])
def test_append(dt, heads_first, tokens, hq, hk, dim, rot, page, interleaved, norm):
    nf4 = lib()
    q, k, v, pos, qw, kw = inputs(tokens, hq, hk, dim, dt, tokens + dim, 3000)
    t = nf4.nf4_rope_table(3000, rot)
    pages = -(-tokens // page) + 3
    shape = (pages, hk, page, dim) if heads_first else (pages, page, hk, dim)
    kc, vc = (torch.randn(shape, device="cuda", generator=gen(s)).to(dt) for s in (1, 2))
    before = kc.clone(), vc.clone()

    def view(c):
        return c.transpose(1, 2) if heads_first else c
    slots = torch.randperm(pages * page, device="cuda", generator=gen(3))[:tokens].contiguous()
    slots[2::5] = -1
    if tokens > 2:
        slots[2] = -(1 << 62)
    out = nf4.nf4_kv_append(view(kc), view(vc), slots, k, v, pos, t, q=q if hq else None, q_weight=qw if norm else None,
                            k_weight=kw if norm else None, interleaved=interleaved)
    cos, sin = angles(pos, frequencies(rot))
    if hq:
        check(out, expected(q, qw if norm else None, cos, sin, interleaved, 1e-6), "q")
    else:
        assert out is None
    real = slots >= 0
    at = slots[real]
    rows = view(kc)[at // page, at % page]
    y, mag = expected(k, kw if norm else None, cos, sin, interleaved, 1e-6)
    check(rows, (y[real], mag[real]), "k")
    assert torch.equal(view(vc)[at // page, at % page], v[real])
    # the rest of both caches is untouched
    for c, b in zip((kc, vc), before):
        other = torch.ones(pages, page, dtype=torch.bool, device="cuda")
        other[at // page, at % page] = False
        assert torch.equal(view(c)[other], view(b)[other])
    assert nf4.nf4_device_error_flags() == 0


@pytest.mark.parametrize("dim", [64, 36])
def test_append_slot_and_position_out_of_range(dim):
    nf4 = lib()
    q, k, v, pos, _, _ = inputs(6, 2, 2, dim, torch.float16, 3, 50)
    t = nf4.nf4_rope_table(50, 16)
    kc = torch.zeros(3, 8, 2, dim, dtype=torch.float16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.tensor([0, 24, 5, 1 << 33, 7, 23], device="cuda")
    out = nf4.nf4_kv_append(kc, vc, slots, k, v, pos, t, q=q)
    assert nf4.nf4_device_error_flags() == 2
    cos, sin = angles(pos, frequencies(16))
    check(out, expected(q, None, cos, sin, False, 0.0), "q")
    written = {0, 5, 7, 23}
    flat = vc.view(24, 2, dim)
    for s in range(24):
        row = [i for i in range(6) if int(slots[i]) == s]
        assert torch.equal(flat[s], v[row[0]] if s in written else torch.zeros_like(flat[s])), s
    pos[2] = 50
    nf4.nf4_kv_append(kc, vc, slots[[0, 4, 2, 5]].contiguous(), k[:4], v[:4], pos[:4].contiguous(), t)
    assert nf4.nf4_device_error_flags() == 2
    assert kc.view(24, 2, dim)[5].isnan().all() and torch.equal(vc.view(24, 2, dim)[5], v[2])
    # no pages at all: every slot is out of range
    nf4.nf4_kv_append(kc[:0], vc[:0], slots, k, v, pos.clamp(max=49), t)
    assert nf4.nf4_device_error_flags() == 2


def test_append_past_32_bits():
    """A cache whose last page lies beyond 2^32 elements, and slots beyond 2^32 in a sparse one."""
    nf4 = lib()
    pages, page, hk, dim = 3, 4, 2, 64
    stride = (1 << 31) + 64
    buf = torch.zeros(2 * stride + page * hk * dim, dtype=torch.bfloat16, device="cuda")
    c = buf.as_strided((pages, page, hk, dim), (stride, hk * dim, dim, 1))
    q, k, v, pos, _, _ = inputs(3, 1, hk, dim, torch.bfloat16, 4, 50)
    t = nf4.nf4_rope_table(50, dim)
    slots = torch.tensor([11, 0, 6], device="cuda")
    v_cache = torch.zeros(pages, page, hk, dim, dtype=torch.bfloat16, device="cuda")
    nf4.nf4_kv_append(c, v_cache, slots, k, v, pos, t)
    _, want = nf4.nf4_qk_norm_rope(q, k, pos, t)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(c[s // page, s % page], want[i])
    assert int(torch.count_nonzero(c)) == int(torch.count_nonzero(want))
    del buf, c
    # 2^17 pages of 2^16 slots that all share one page's memory (page stride 0)
    one = torch.zeros(1, 65536, 1, 8, dtype=torch.bfloat16, device="cuda")
    wide = one.expand(1 << 17, 65536, 1, 8)
    x = torch.randn(2, 1, 8, device="cuda").bfloat16()
    slots = torch.tensor([(1 << 32) + 65536 * 5 + 123, 77], device="cuda")
    nf4.nf4_kv_append(wide, torch.zeros_like(one).expand(1 << 17, 65536, 1, 8), slots, x, x,
                      torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(1, 0, 2, device="cuda"))
    assert torch.equal(one[0, 123, 0], x[0, 0]) and torch.equal(one[0, 77, 0], x[1, 0])
    assert nf4.nf4_device_error_flags() == 0


def test_empty_calls():
    nf4 = lib()
    t = nf4.nf4_rope_table(4, 8)
    e = torch.empty(0, 2, 8, dtype=torch.bfloat16, device="cuda")
    p = torch.empty(0, dtype=torch.int64, device="cuda")
    q, k = nf4.nf4_qk_norm_rope(e, e, p, t)
    assert q.shape == e.shape and k.shape == e.shape
    c = torch.zeros(2, 4, 2, 8, dtype=torch.bfloat16, device="cuda")
    assert nf4.nf4_kv_append(c, c.clone(), p, e, e, p, t) is None
    assert nf4.nf4_rope_table(0, 8).shape == (0, 4, 2)

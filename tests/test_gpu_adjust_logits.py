"""nf4_adjust_logits against its documented steps, each a binary32 operation rounded to nearest, done by
numpy: results are equal bit for bit (NaN apart from its payload); and against binary64.

Tolerance against binary64: the division or product, f c, the two differences, the bias sum of m entries and
its addition are at most 5 + m roundings of 2^-24, each relative to a value of at most
M = |x| max(rho, 1 / rho) + f c + p + sum |bias|; the result is rounded once (half a step: 2^-8 in bf16,
2^-11 in fp16, 2^-24 in fp32)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}


def lib():
    import w4a16_gemv_gb300 as nf4
    return nf4


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Inputs on the host (numpy) and on the GPU. counts: rows of each request."""

    def __init__(self, counts, vocab, dtype, seed=0, history=50, bias=6, mask=True, draft=True, penalties=True, pad=0):
        rng = np.random.default_rng(seed)
        self.counts, self.vocab, self.dtype = counts, vocab, dtype
        rows, requests = sum(counts), len(counts)
        self.cu = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
        wide = torch.from_numpy(rng.normal(0, 3, (rows, vocab + pad)).astype(np.float32)).to(DTYPES[dtype]).cuda()
        self.logits = wide[:, :vocab]
        self.kw = {"cu_rows": on_gpu(self.cu)}
        self.h = {}

        def put(name, value):
            self.h[name] = value
            self.kw[name] = on_gpu(value)

        if history is not None:
            put("history", np.minimum(vocab ** rng.random((requests, history)), vocab - 1).astype(np.int32))
            put("history_lens", rng.integers(0, history + 1, requests).astype(np.int32))
            put("prompt_lens", rng.integers(0, history + 1, requests).astype(np.int32))
        if penalties:
            put("repetition", (1 + rng.random(requests) * 0.5).astype(np.float32))
            put("frequency", (rng.random(requests) - 0.3).astype(np.float32))
            put("presence", (rng.random(requests) - 0.3).astype(np.float32))
        if bias is not None:
            put("bias_tokens", rng.integers(-2, vocab, (requests, bias)).astype(np.int32))
            if bias > 2:
                self.h["bias_tokens"][:, 2] = self.h["bias_tokens"][:, 0]  # the same token twice
            put("bias_tokens", self.h["bias_tokens"])
            put("bias_values", (rng.normal(0, 4, (requests, bias))).astype(np.float32))
        if mask:
            put("mask", rng.integers(-2 ** 31, 2 ** 31, (requests + 1, (vocab + 31) // 32)).astype(np.int32))
            put("mask_rows", rng.integers(-1, requests + 1, rows).astype(np.int32))
        if draft:
            put("draft_tokens", rng.integers(0, vocab, rows).astype(np.int32))
            bits = -(-max(counts + [1]) // 64)
            put("tree_mask", rng.integers(-2 ** 63, 2 ** 63, (rows, bits)).astype(np.int64))

    def context(self, r):
        """The request of row r (or None), and per token how often it stands in the answer and whether it is known."""
        count, known = np.zeros(self.vocab, np.int64), np.zeros(self.vocab, bool)
        b = next((b for b, n in enumerate(self.counts) if self.cu[b] <= r < self.cu[b] + n), None)
        if b is None:
            return None, count, known
        if "history" in self.h:
            words = self.h["history"][b, :self.h["history_lens"][b]]
            prompt = self.h["prompt_lens"][b] if "prompt_lens" in self.h else 0
            np.add.at(count, words[prompt:], 1)
            known[words] = True
        if "draft_tokens" in self.h:
            for x in range(min(self.counts[b], 64 * self.h["tree_mask"].shape[1])):
                if int(self.h["tree_mask"][r, x // 64]) >> (x % 64) & 1:
                    v = self.h["draft_tokens"][self.cu[b] + x]
                    count[v] += 1
                    known[v] = True
        return b, count, known

    def want(self, r, t=np.float32):
        """Row r in steps of type t, before the rounding; and the sum of absolute values in binary64."""
        b, count, known = self.context(r)
        x = self.logits[r].float().cpu().numpy().astype(t)
        size = np.abs(x.astype(np.float64))
        with np.errstate(all="ignore"):
            if b is not None:
                rho, f, p = (t(self.h[n][b]) if n in self.h else t(d) for n, d in
                             (("repetition", 1), ("frequency", 0), ("presence", 0)))
                x = np.where(known, np.where(x > 0, x / rho, x * rho), x).astype(t)
                size = size * max(rho, 1 / rho) + abs(float(f)) * count + abs(float(p))
                x = np.where(count > 0, (x - (f * count.astype(t)).astype(t)).astype(t) - p, x).astype(t)
                if "bias_tokens" in self.h:
                    total, has = np.zeros(self.vocab, t), np.zeros(self.vocab, bool)
                    for v, y in zip(self.h["bias_tokens"][b], self.h["bias_values"][b]):
                        if 0 <= v < self.vocab:
                            total[v] = total[v] + t(y)
                            has[v] = True
                            size[v] += abs(float(y))
                    x = np.where(has, x + total, x).astype(t)
            if "mask" in self.h:
                m = self.h["mask_rows"][r] if "mask_rows" in self.h else r
                if 0 <= m < self.h["mask"].shape[0]:
                    v = np.arange(self.vocab)
                    x = np.where(self.h["mask"][m][v // 32] >> (v % 32) & 1, x, t("-inf")).astype(t)
        return x, size

    def run(self, **kw):
        kw.setdefault("return_best", True)
        return lib().nf4_adjust_logits(self.logits, **{**self.kw, **kw})

    def check(self, got, rows=None, close=True):
        out, best = got
        assert out.dtype == DTYPES[self.dtype] and best.dtype == torch.int32
        for r in rows if rows is not None else range(out.shape[0]):
            want = torch.from_numpy(self.want(r)[0]).to(out.dtype)
            have = out[r].cpu()
            same = (want == have) | (want.isnan() & have.isnan())
            assert same.all(), (r, (~same).nonzero()[:5, 0].tolist(), have[~same][:5], want[~same][:5])
            f = have.float().numpy()
            first = int(np.flatnonzero(np.isnan(f))[0]) if np.isnan(f).any() else int(np.argmax(f))
            assert int(best[r]) == first, (r, int(best[r]), first)
            if close:
                x, size = self.want(r, np.float64)
                fin = np.isfinite(x)
                m = self.h["bias_tokens"].shape[1] if "bias_tokens" in self.h else 0
                err = np.abs(have.double().numpy()[fin] - x[fin])
                tol = U[self.dtype] * np.abs(x[fin]) + (5 + m) * 2.0 ** -24 * size[fin] * (1 + U[self.dtype]) + 2.0 ** -24
                assert (err <= tol).all(), r


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("counts,vocab", [([1], 1), ([1, 1], 7), ([1], 32), ([3, 1], 65), ([1, 0, 2], 1000), ([5, 70], 4099),
                                          ([2, 1], 32001), ([1, 3], 100003)])
def test_everything_at_once(dtype, counts, vocab):
    c = Case(counts, vocab, dtype, seed=vocab)
    got = c.run()
    c.check(got)
    again = c.run()
    assert torch.equal(got[0].view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(got[1], again[1])
    assert lib().nf4_device_error_flags() == 0


@pytest.mark.parametrize("bias", [1, 3, 5, 7, 33, 1023])
@pytest.mark.parametrize("history", [None, 1, 235, 3000])
def test_bias_lists_of_any_length(bias, history):
    """(what lies behind the list in shared memory is read 16 bytes at a time)"""
    c = Case([1] * 9 + [6], 1307, "bf16" if bias % 4 == 1 else "fp32", seed=bias, history=history, bias=bias)
    c.check(c.run(), close=bias < 100)
    assert lib().nf4_device_error_flags() == 0


def test_logits_and_outputs_are_columns_of_one_buffer():
    c = Case([1, 3], 500, "bf16", seed=12)
    want = c.run()
    both = torch.cat((c.logits, torch.zeros_like(c.logits)), 1)
    c.logits = both[:, :500]
    got = c.run(out=both[:, 500:])
    assert torch.equal(got[0].view(torch.int16), want[0].view(torch.int16)) and torch.equal(got[1], want[1])
    with pytest.raises(lib().NF4Error, match="INVALID_SIZE"):
        c.run(out=both[:, 499:999])


@pytest.mark.parametrize("parts", [dict(history=None), dict(bias=None), dict(mask=False), dict(draft=False),
                                   dict(penalties=False), dict(history=None, draft=False), dict(history=None, bias=None, draft=False),
                                   dict(history=None, bias=None, draft=False, mask=False, penalties=False),
                                   dict(history=0, bias=0)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_parts(parts, dtype):
    for counts, vocab in (([1, 4, 2], 5000), ([1], 70000)):
        c = Case(counts, vocab, dtype, seed=9, **parts)
        c.check(c.run())
    assert lib().nf4_device_error_flags() == 0


@pytest.mark.parametrize("vocab", [400001, 1000003])
def test_vocabularies_of_several_passes(vocab):
    c = Case([2, 1], vocab, "bf16", seed=2, history=3000)
    c.check(c.run(), close=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_histories_and_many_rows(dtype):
    c = Case([1] * 150 + [33, 64], 3001, dtype, seed=3, history=20000, bias=300)
    c.check(c.run(), rows=[0, 77, 149, 150, 182, 183, 246])
    one = Case([1], 50000, dtype, seed=4, history=100000, bias=1024)
    one.h["bias_tokens"][:] = np.arange(1024) % 500
    one.kw["bias_tokens"] = on_gpu(one.h["bias_tokens"])
    one.check(one.run(), close=False)


def test_one_token_many_times():
    """Counts far past 16 bits, from all CTAs of a cluster to one word."""
    c = Case([1], 20000, "fp32", seed=5, history=200000, draft=False)
    c.h["history"][:] = 12345
    c.h["history_lens"][:], c.h["prompt_lens"][:] = 200000, 3
    c.h["frequency"][:] = 2.0 ** -10
    for n in ("history", "history_lens", "prompt_lens", "frequency"):
        c.kw[n] = on_gpu(c.h[n])
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad", [0, 1, 3, 8])
def test_strides_and_outputs(dtype, pad):
    """Rows apart; outputs whose rows are and are not alike modulo 16 bytes; in place."""
    c = Case([2, 1, 3], 9001, dtype, seed=pad, pad=pad)
    want, best = c.run()
    c.check((want, best))
    for offset in (0, 1, 5):
        wide = torch.full((6, 9001 + offset + 7), 7.0, dtype=want.dtype, device="cuda")
        out = wide[:, offset:offset + 9001]
        got, b = c.run(out=out)
        assert got is out and torch.equal(got, want) and torch.equal(b, best)
        assert (wide[:, :offset] == 7).all() and (wide[:, offset + 9001:] == 7).all()
    keep = c.logits.clone()
    out, b = c.run(out=c.logits)
    assert torch.equal(out, want) and torch.equal(b, best) and out.data_ptr() == c.logits.data_ptr()
    c.logits.copy_(keep)
    into = torch.empty(6, dtype=torch.int32, device="cuda")
    assert c.run(best=into)[1] is into and torch.equal(into, best)
    assert torch.equal(c.run(return_best=False), want)


def test_rows_that_no_request_holds():
    c = Case([2, 0, 3], 2000, "fp32", seed=1)
    rows = 9
    wide = torch.randn(rows, 2000, device="cuda")
    wide[2:7] = c.logits
    c.logits = wide
    c.cu = c.cu + 2
    c.h["mask_rows"] = np.array([0, -1, 1, 2, -1, 3, 0, 1, -1], np.int32)
    c.h["draft_tokens"] = np.random.default_rng(1).integers(0, 2000, rows).astype(np.int32)
    c.h["tree_mask"] = np.random.default_rng(2).integers(-2 ** 63, 2 ** 63, (rows, 1)).astype(np.int64)
    for n in ("mask_rows", "draft_tokens", "tree_mask"):
        c.kw[n] = on_gpu(c.h[n])
    c.kw["cu_rows"] = on_gpu(c.cu)
    c.check(c.run())
    assert lib().nf4_device_error_flags() == 0


def test_no_requests_at_all():
    c = Case([], 100, "fp32", mask=False, draft=False)
    c.logits = torch.randn(4, 100, device="cuda")
    out, best = lib().nf4_adjust_logits(c.logits, cu_rows=on_gpu(np.zeros(1, np.int32)), return_best=True,
                                        history=torch.zeros(0, 3, dtype=torch.int32, device="cuda"),
                                        history_lens=torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert torch.equal(out, c.logits) and torch.equal(best.long(), c.logits.argmax(1))
    empty = lib().nf4_adjust_logits(c.logits[:0], return_best=True)
    assert empty[0].shape == (0, 100) and empty[1].shape == (0,)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_best_of_ties_and_non_finite_values(dtype):
    nan, inf = float("nan"), float("inf")
    rows = [[1.0, 3.0, 3.0, 2.0], [-0.0, 0.0, -1.0, 0.0], [nan, 1.0, nan, inf], [1.0, inf, -inf, inf], [-inf] * 4,
            [-2.0, -1.0, -1.0, -5.0], [1.0, nan, nan, 2.0], [-nan, 1.0, 0.0, 2.0]]
    want = [1, 0, 0, 1, 0, 1, 1, 0]
    x = torch.zeros(len(rows), 30011, dtype=DTYPES[dtype], device="cuda").fill_(-inf)
    for at in (0, 5, 4096, 20000, 30007):
        y = x.clone()
        y[:, at:at + 4] = torch.tensor(rows).to(y.dtype).cuda()
        out, best = lib().nf4_adjust_logits(y, return_best=True)
        assert torch.equal(out.view(torch.uint8), y.view(torch.uint8))
        assert best.tolist() == [w + at if w or rows[i] != [-inf] * 4 else 0 for i, w in enumerate(want)], at


def test_non_finite_logits_and_masks():
    """A masked token is -infinity whatever stood there; nothing masked leaves NaN alone; all masked: best 0."""
    x = torch.randn(3, 5000, device="cuda")
    x[:, 10], x[:, 11], x[:, 12] = float("nan"), float("inf"), float("-inf")
    mask = torch.full((2, 157), -1, dtype=torch.int32, device="cuda")
    mask[0, 0] = ~(7 << 10)
    mask[1] = 0
    rows = torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda")
    kw = dict(history=torch.tensor([[10, 11, 12, 12]] * 3, dtype=torch.int32, device="cuda"),
              history_lens=torch.tensor([4] * 3, dtype=torch.int32, device="cuda"),
              repetition=torch.full((3,), 1.3, device="cuda"), presence=torch.ones(3, device="cuda"))
    out, best = lib().nf4_adjust_logits(x, mask=mask, mask_rows=rows, return_best=True, **kw)
    assert (out[0, 10:13] == float("-inf")).all() and torch.equal(out[0, 13:], x[0, 13:])
    assert (out[1] == float("-inf")).all() and int(best[1]) == 0
    assert out[2, 10].isnan() and out[2, 11] == float("inf") and out[2, 12] == float("-inf") and int(best[2]) == 10
    assert int(best[0]) == int(out[0].argmax())
    lowest = torch.full((1, 64), torch.finfo(torch.float32).min, device="cuda")
    out, best = lib().nf4_adjust_logits(lowest, mask=torch.tensor([[0, 8]], dtype=torch.int32, device="cuda"), return_best=True)
    assert int(best[0]) == 35 and float(out[0, 35]) == torch.finfo(torch.float32).min


def test_values_out_of_range_are_not_counted_and_reported():
    c = Case([1, 1], 1000, "fp32", seed=6, draft=False)
    want = c.run()
    h = torch.cat((c.kw["history"], torch.zeros(2, 3, dtype=torch.int32, device="cuda")), 1)
    lens = c.kw["history_lens"].clone()
    for b in range(2):  # tokens that do not exist, at the end of the history
        h[b, lens[b]:lens[b] + 3] = torch.tensor([-1, 1000, 1 << 30])
    got = c.run(history=h, history_lens=lens + 3)
    assert torch.equal(got[0], want[0]) and lib().nf4_device_error_flags() == 2
    t = c.kw["bias_tokens"].clone()
    t[:, 5] = -1
    want = c.run(bias_tokens=t)
    t[:, 5] = 1000
    assert torch.equal(c.run(bias_tokens=t)[0], want[0]) and lib().nf4_device_error_flags() == 2
    m = c.kw["mask_rows"].clone()
    m[0] = -1
    want = c.run(mask_rows=m)
    m[0] = 3
    assert torch.equal(c.run(mask_rows=m)[0], want[0]) and lib().nf4_device_error_flags() == 2
    full = torch.full_like(lens, 50)
    want = c.run(history_lens=full)
    assert torch.equal(c.run(history_lens=full * 10)[0], want[0]) and lib().nf4_device_error_flags() == 2
    cu = torch.tensor([-3, 1, 99], dtype=torch.int32, device="cuda")
    want = c.run()
    assert torch.equal(c.run(cu_rows=cu)[0], want[0]) and lib().nf4_device_error_flags() == 2


def test_recorded_beside_another_stream():
    c = Case([4, 1, 7], 20011, "bf16", seed=8)
    want = c.run()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, best = c.run()
        for _ in range(4):
            graph.replay()
            again = c.run(stream=other)
    torch.cuda.synchronize()
    for o, b in ((out, best), again):
        assert torch.equal(o, want[0]) and torch.equal(b, want[1])


def test_refusals():
    x = torch.randn(2, 100, device="cuda")
    i = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    run = lib().nf4_adjust_logits
    for kw, error, match in ((dict(history=i), TypeError, "together"), (dict(bias_tokens=i), TypeError, "together"),
                             (dict(draft_tokens=i[:, 0]), TypeError, "together"), (dict(mask_rows=i[:, 0]), TypeError, "mask"),
                             (dict(mask=i), ValueError, "shape"),
                             (dict(mask=torch.zeros(3, 4, dtype=torch.int32, device="cuda")), ValueError, "row for each"),
                             (dict(repetition=torch.ones(3, device="cuda")), ValueError, "shape"),
                             (dict(repetition=torch.ones(2, device="cuda").double()), TypeError, "float32"),
                             (dict(out=torch.empty(2, 100, device="cuda").bfloat16()), TypeError, "float32"),
                             (dict(out=torch.empty(1, 100, device="cuda").expand(2, 100)), lib().NF4Error, "INVALID_SIZE"),
                             (dict(cu_rows=torch.zeros(0, dtype=torch.int32, device="cuda")), ValueError, "cu_rows"),
                             (dict(history=i.long(), history_lens=i[:, 0].contiguous()), TypeError, "int32"),
                             (dict(bias_tokens=torch.zeros(2, 1025, dtype=torch.int32, device="cuda"),
                                   bias_values=torch.zeros(2, 1025, device="cuda")), lib().NF4Error, "INVALID_SIZE")):
        with pytest.raises(error, match=match):
            run(x, **kw)
    with pytest.raises(TypeError, match="bf16, fp16 or fp32"):
        run(x.double())


def layout(c, rows, offset):
    """Random logits for the case, their rows on 16-byte boundaries ("aligned"), at the same distance from one ("alike": an
    odd row length is not a whole number of chunks) or one after another ("dense"); and an output laid out alike."""
    dtype, vocab = DTYPES[c.dtype], c.vocab
    stride = vocab if offset is None else -(-vocab // 8) * 8 + 8
    at = offset or 0
    g = torch.Generator(device="cuda")
    g.manual_seed(rows)
    wide = (torch.randn(2, rows, stride, device="cuda", generator=g) * 3).to(dtype)
    c.logits = wide[0, :, at:at + vocab]
    return wide[1, :, at:at + vocab]


def forest(counts, vocab, dtype, history, offset, gap=(0, 0), pool=24, seed=0, bias=5):
    """A case of many rows whose drafted tokens are few different ones, side by side in pairs, so that the branches of
    neighbouring rows share tokens and words; the histories hold some of them. gap: rows before and behind the requests'."""
    c = Case(counts, vocab, dtype, seed=seed, history=history, bias=bias)
    rng = np.random.default_rng(seed + 1)
    rows = sum(counts) + sum(gap)
    first = rng.integers(0, vocab // 2, pool // 2) * 2
    tokens = np.concatenate((first, first + 1)).astype(np.int32)
    c.cu = c.cu + np.int32(gap[0])
    c.h["draft_tokens"] = rng.choice(tokens, rows).astype(np.int32)
    c.h["tree_mask"] = rng.integers(-2 ** 63, 2 ** 63, (rows, c.h["tree_mask"].shape[1])).astype(np.int64)
    c.h["mask_rows"] = rng.integers(-1, c.h["mask"].shape[0], rows).astype(np.int32)
    c.h["history"][:, ::5] = rng.choice(tokens, c.h["history"][:, ::5].shape)
    for n in ("draft_tokens", "tree_mask", "mask_rows", "history"):
        c.kw[n] = on_gpu(c.h[n])
    c.kw["cu_rows"] = on_gpu(c.cu)
    return c, layout(c, rows, offset)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab,offset", [(1000, 0), (1003, 0), (1003, 3), (1003, None)], ids=["aligned", "odd", "skewed", "dense"])
def test_many_rows_in_trees(dtype, vocab, offset):
    """More rows than there are CTAs (two on each of 152 SMs), so that a cluster takes several: from branch to branch of a
    request, from request to request, and rows that no request holds before and behind them."""
    counts = [1, 7, 40, 70, 0] * 6
    c, out = forest(counts, vocab, dtype, 50, offset, gap=(5, 9), seed=vocab)
    got = c.run()
    c.check(got)
    into, best = c.run(out=out)  # rows alike in input and output, 16 bytes at a time
    assert into is out and torch.equal(into, got[0]) and torch.equal(best, got[1])
    into, best = c.run(out=c.logits)
    assert into is c.logits and torch.equal(into, got[0]) and torch.equal(best, got[1])
    assert lib().nf4_device_error_flags() == 0


@pytest.mark.parametrize("dtype,history", [("bf16", 50), ("fp16", 20000), ("fp32", 300), ("fp32", 20000)])
@pytest.mark.parametrize("vocab,offset", [(20000, 0), (20003, 2)], ids=["aligned", "skewed"])
def test_many_rows_of_several_ctas(dtype, history, vocab, offset):
    """Clusters of four CTAs (74 at once, or fewer) with several rows each; words of 16 bits and, for histories past their
    counts, of 32."""
    counts = [3, 70, 1, 40, 100, 7]
    c, out = forest(counts, vocab, dtype, history, offset, seed=history)
    got = c.run(out=out)
    c.check(got, rows=[0, 1, 2, 3, 4, 40, 72, 73, 74, 75, 90, 113, 114, 115, 116, 117, 170, 213, 214, 215, 220], close=False)
    dense = c.run()  # (other offsets of rows modulo 16 bytes)
    assert torch.equal(dense[0], got[0]) and torch.equal(dense[1], got[1])
    assert lib().nf4_device_error_flags() == 0


def test_many_rows_one_each():
    """More requests than 64 rows of every cluster, each with a history of its own."""
    c = Case([1] * 21000, 100, "fp32", seed=2, history=9, bias=3, draft=False)
    rows = list(range(0, 21000, 97)) + [20999]
    c.check(c.run(), rows=rows, close=False)
    assert lib().nf4_device_error_flags() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_more_tokens_than_the_list_holds(dtype):
    """Every token of a vocabulary in the history: 15000 of each of eight CTAs, whose lists hold 8192."""
    c = Case([1], 120000, dtype, seed=4, history=200000, draft=False)
    rng = np.random.default_rng(5)
    c.h["history"][0] = np.concatenate((rng.permutation(120000), rng.integers(0, 120000, 80000)))
    c.h["history_lens"][:], c.h["prompt_lens"][:] = 200000, 100000
    for n in ("history", "history_lens", "prompt_lens"):
        c.kw[n] = on_gpu(c.h[n])
    c.check(c.run(), close=False)
    assert lib().nf4_device_error_flags() == 0


@pytest.mark.parametrize("words", [8191, 8180, 16000])
def test_lists_that_fill_up(words):
    """So many words of one CTA's blocks (those are dealt out in turn, 256 tokens each, to four) that its list is full, or
    becomes full as the branches of a tree bring tokens to it."""
    vocab, counts = 70000, [20] * 8
    c, out = forest(counts, vocab, "bf16", words, 0, seed=words, pool=2)
    mine = np.flatnonzero(np.arange(vocab) // 256 % 4 == 1)
    rng = np.random.default_rng(words)
    for b in range(len(counts)):
        c.h["history"][b] = rng.permutation(mine)[:words]
    c.h["history_lens"][:], c.h["prompt_lens"][:] = words, words // 2
    c.h["draft_tokens"][:] = rng.choice(mine, len(c.h["draft_tokens"]))
    for n in ("history", "history_lens", "prompt_lens", "draft_tokens"):
        c.kw[n] = on_gpu(c.h[n])
    c.check(c.run(out=out), rows=range(0, 160, 3), close=False)
    assert lib().nf4_device_error_flags() == 0


def test_offsets_past_32_bits():
    """5 G bytes of logits: the last rows are as the same rows by themselves."""
    rows, vocab, last = 40000, 64001, 25
    x = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    x.normal_()
    c = Case([last], vocab, "bf16", seed=1)
    x[-last:] = c.logits
    cu = torch.tensor([rows - last, rows], dtype=torch.int32, device="cuda")
    kw = {k: v for k, v in c.kw.items() if k not in ("cu_rows", "draft_tokens", "tree_mask", "mask_rows")}
    draft = torch.zeros(rows, dtype=torch.int32, device="cuda")
    tree = torch.zeros(rows, 1, dtype=torch.int64, device="cuda")
    mask_rows = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    draft[-last:], tree[-last:], mask_rows[-last:] = c.kw["draft_tokens"], c.kw["tree_mask"], c.kw["mask_rows"]
    out, best = lib().nf4_adjust_logits(x, cu_rows=cu, draft_tokens=draft, tree_mask=tree, mask_rows=mask_rows, return_best=True, **kw)
    assert torch.equal(out[:-last], x[:-last])
    for r in range(0, rows - last, 4999):
        assert int(best[r]) == int((x[r] == x[r].max()).nonzero()[0])
    c.check((out[-last:], best[-last:]), close=False)
    assert lib().nf4_device_error_flags() == 0


def test_calls_on_several_streams():
    """Calls that run beside one another on the same inputs."""
    c = Case([20, 70, 1], 50003, "bf16", seed=2, history=3000)
    want = c.run()
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [c.run(stream=streams[i % 4]) for i in range(24)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(b, want[1]) for o, b in got)

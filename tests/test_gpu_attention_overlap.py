"""Attention calls that overlap others in time, in one stream and in two, never synchronised in between: every output is
bit for bit what the call gives alone."""
import pytest
import torch

from test_gpu_prefix_attention import Call, lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
def test_beside_kernels_that_take_tensor_memory(dim):
    """Attention and the tensor-core GEMV in turn in two streams: both hold tensor memory, and each starts while the one
    before it still runs."""
    nf4 = lib()
    code2 = torch.tensor([(i - 127.5) / 127.5 for i in range(256)], dtype=torch.float16, device="cuda")
    wt = nf4.nf4_quantize(torch.randn(1024, 1024, device="cuda") * 0.02, code2)
    x = torch.randn(32, 1024, device="cuda").bfloat16()
    y = nf4.gemv(wt, x)
    calls = [Call(8, 2, dim, prefix, [100 + 5 * b for b in range(n)], [1] * n, seed=prefix) for prefix, n in
             ((4000, 40), (9000, 3))]
    calls.append(Call(8, 2, dim, 700, [300, 200], [300, 150], seed=2))  # the own items join the shared ones
    calls.append(Call(8, 2, dim, 700, [0], [70], width=0, seed=3))      # one launch
    want = [c.run() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(100):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                n = (i + k) % len(calls)
                got.append((n, *calls[n].run(), nf4.gemv(wt, x)))
    torch.cuda.synchronize()
    for n, out, lse, z in got:
        assert torch.equal(out, want[n][0]) and torch.equal(lse, want[n][1]) and torch.equal(z, y)
    assert nf4.nf4_device_error_flags() == 0


@pytest.mark.parametrize("dim,rot", [(128, 128), (80, 40), (36, 18)], ids=["16 bytes", "8 bytes", "elements"])
def test_what_the_launch_before_has_just_written(dim, rot):
    """The table, the rows and the norm's weights of a call are the outputs of the ones right before it, in the same
    buffers every time."""
    nf4 = lib()
    tokens, heads = 300, 6
    pos = torch.randint(0, 500, (tokens,), device="cuda")
    x = torch.randn(tokens, heads, dim, device="cuda").bfloat16()
    one = torch.zeros(1, dtype=torch.int64, device="cuda")
    table, q, k, kk, w = (torch.empty(s, dtype=t, device="cuda") for s, t in (
        ((500, rot // 2, 2), torch.float32), (x.shape, x.dtype), (x.shape, x.dtype), (x.shape, x.dtype),
        ((1, 1, dim), x.dtype)))

    def step(i, wait):
        nf4.nf4_rope_table(500, rot, base=100.0 + 50 * i, out=table)
        wait()
        # rotated weights, and rows rotated by the new table
        nf4.nf4_qk_norm_rope(x[i:i + 1, :1], x[i:i + 1, 1:2], one + i, table, q_out=w, k_out=kk[:1, :1])
        wait()
        nf4.nf4_qk_norm_rope(x, x, pos, table, q_weight=w[0, 0], q_out=q, k_out=k)
        wait()
        nf4.nf4_qk_norm_rope(q, k, pos, table, k_weight=w[0, 0], q_out=q, k_out=kk)
        wait()
        return q.clone(), kk.clone()

    want = [step(i, torch.cuda.synchronize) for i in range(20)]
    got = [step(i, lambda: None) for _ in range(5) for i in range(20)]
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(got):
        assert torch.equal(a, want[i % 20][0]) and torch.equal(b, want[i % 20][1])
    assert nf4.nf4_device_error_flags() == 0


@pytest.mark.parametrize("dim", [128, 24])
def test_tokens_that_go_nowhere_beside_others(dim):
    """Appends of nothing but padding leave the cache as it is, and disturb no call that takes their place on the SMs."""
    nf4 = lib()
    tokens, heads = 2000, 8
    pos = torch.randint(0, 500, (tokens,), device="cuda")
    table = nf4.nf4_rope_table(500, dim)
    x = torch.randn(tokens, heads, dim, device="cuda").bfloat16()
    cache = torch.randn(3, 16, heads, dim, device="cuda").bfloat16()
    kept = cache.clone()
    none = torch.full((tokens,), -1, device="cuda")
    want = nf4.nf4_qk_norm_rope(x, x, pos, table)[0].clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(50):
        for s in streams:
            with torch.cuda.stream(s):
                nf4.nf4_kv_append(cache, cache, none, x, x, pos, table)
                got.append(nf4.nf4_qk_norm_rope(x, x, pos, table)[0])
    torch.cuda.synchronize()
    assert torch.equal(cache, kept) and all(torch.equal(g, want) for g in got)
    assert nf4.nf4_device_error_flags() == 0


def test_calls_that_follow_one_another_through_one_workspace():
    """Steps of an append and an attention over it, of three plans (own keys joined on the way out, two launches and a join,
    one launch) and two values of every input, never synchronised: first through one workspace in one stream, then in two
    streams with one each. A part read before it is written, or overwritten before it is read, is another call's."""
    nf4 = lib()
    cases = []
    for prefix, counts, lens in ((700, [300, 150], [300, 200]), (6000, [1] * 40, [90 + b for b in range(40)]),
                                 (500, [60], [0])):
        for seed in (1, 2):
            width = None if lens[0] else 0
            c = Call(8, 2, 128, prefix, lens, counts, seed=seed, junk=0.25, width=width)
            tokens = sum(counts)
            new = torch.randn(tokens, 12, 128, device="cuda").bfloat16()
            table = nf4.nf4_rope_table(100, 128, base=50.0 * seed)
            pos = torch.randint(0, 100, (tokens,), device="cuda")
            # every token's key and value go to its sequence's last slots, or nowhere
            slots = []
            for b, (n, m) in enumerate(zip(counts, lens)):
                at = [m - n + i for i in range(n)]
                slots += [int(c.suffix_pages[b, j // c.page]) * c.page + j % c.page if m else -1 for j in at]
            cases.append((c, new, table, pos, torch.tensor(slots, device="cuda")))
    need = max(nf4.nf4_prefix_attention_workspace_size(*c.args(), cu_q=c.cu_q) for c, *_ in cases)

    def step(n, ws):
        c, new, table, pos, slots = cases[n]
        q = nf4.nf4_kv_append(c.k, c.v, slots, new[:, 8:10], new[:, 10:], pos, table, q=new[:, :8])
        return nf4.nf4_prefix_attention(q, *c.args()[1:], cu_q=c.cu_q, return_lse=True, workspace=ws)

    spaces = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = []
    for n in range(len(cases)):
        want.append(step(n, spaces[0]))
        torch.cuda.synchronize()
    # (in two streams, each keeps to cases of its own: an append writes the cache that its call reads)
    for parts in ([list(range(6))], [[0, 2, 4], [1, 3, 5]]):
        streams = [torch.cuda.Stream() for _ in parts]
        got = []
        for i in range(60):
            for k, (mine, s) in enumerate(zip(parts, streams)):
                with torch.cuda.stream(s):
                    n = mine[i * 5 % len(mine)]
                    got.append((n, *step(n, spaces[k])))
        torch.cuda.synchronize()
        for n, out, lse in got:
            assert torch.equal(out, want[n][0]) and torch.equal(lse, want[n][1]), n
    assert nf4.nf4_device_error_flags() == 0

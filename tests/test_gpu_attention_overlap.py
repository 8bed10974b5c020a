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

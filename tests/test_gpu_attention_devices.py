"""Tensors on a device other than the call's are refused. The other device is made up (a tensor without memory), so
that one GPU is enough and nothing could be read or written there."""
import pytest
import torch

pytestmark = pytest.mark.gpu


class Elsewhere(torch.Tensor):
    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError("there is no such device")


def elsewhere(*shape, dtype):
    return torch.Tensor._make_wrapper_subclass(Elsewhere, shape, dtype=dtype, device="cuda:7")


def test_attention_workspace():
    import w4a16_gemv_gb300 as nf4
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    args = (q, cache, cache, torch.zeros(2, dtype=torch.int32, device="cuda"), 20,
            torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda"))
    need = nf4.nf4_prefix_attention_workspace_size(*args)
    assert need > 0
    with pytest.raises(ValueError, match="same device"):
        nf4.nf4_prefix_attention(*args, workspace=elsewhere(need, dtype=torch.uint8))
    with pytest.raises(ValueError, match="same device"):
        nf4.nf4_prefix_attention(*args, out=elsewhere(2, 4, 64, dtype=torch.bfloat16))

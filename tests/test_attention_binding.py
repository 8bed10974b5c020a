"""The Python side of the attention binding without a GPU: what reaches the C calls."""
import pytest
import torch


@pytest.fixture(scope="module")
def attention():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import w4a16_gemv_gb300.attention as attention
    return attention


class Table:
    """Stands in for a float32 CUDA tensor of a table."""
    dtype = torch.float32
    is_cuda = True

    def __init__(self, shape, device="cuda:0"):
        self.shape, self.device = torch.Size(shape), torch.device(device)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000


@pytest.fixture
def calls(attention, monkeypatch):
    """nf4_rope_table's argument structures, instead of the call."""
    seen = []

    class Lib:
        @staticmethod
        def nf4_rope_table(args, stream):
            a = args._obj
            seen.append({f: getattr(a, f) for f, _ in a._fields_})
            return 0

    monkeypatch.setattr(attention, "_lib", Lib)
    return seen


@pytest.mark.parametrize("scaling,high", [("bands", 4.0), ("ramp", 32.0)])
def test_rope_table_defaults(attention, calls, scaling, high):
    """The published values: by wavelength 1 and 4 turns, by index 1 and 32."""
    out = Table((64, 16, 2))
    attention.nf4_rope_table(64, 32, scaling=scaling, factor=4.0, out=out, stream=7)
    attention.nf4_rope_table(64, 32, scaling=scaling, factor=4.0, high=9.0, out=out, stream=7)
    assert [(c["low"], c["high"]) for c in calls] == [(1.0, high), (1.0, 9.0)]

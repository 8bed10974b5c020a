"""The Python side of the attention binding without a GPU: what reaches the C calls."""
import os
import shutil
import subprocess
import sys

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

    def numel(self):
        return self.shape.numel()

    def record_stream(self, stream):
        self.kept_for = stream


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream, self.device = handle, device


@pytest.fixture
def calls(attention, monkeypatch):
    """nf4_rope_table's argument structures, the stream and the current device, instead of the call, on a machine
    of two GPUs of which device 0 is current and whose current streams are 100 and 101."""
    seen, current = [], [0]

    class Lib:
        @staticmethod
        def nf4_rope_table(args, stream):
            a = args._obj
            seen.append({**{f: getattr(a, f) for f, _ in a._fields_}, "stream": stream, "device": current[-1]})
            return 0

    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            current.append(self.index)

        def __exit__(self, *_):
            current.pop()

    monkeypatch.setattr(attention, "_lib", Lib)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(100 + current[-1]))
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: Stream(0, device))
    return seen


@pytest.mark.parametrize("scaling,high", [("bands", 4.0), ("ramp", 32.0)])
def test_rope_table_defaults(attention, calls, scaling, high):
    """The published values: by wavelength 1 and 4 turns, by index 1 and 32."""
    out = Table((64, 16, 2))
    attention.nf4_rope_table(64, 32, scaling=scaling, factor=4.0, out=out, stream=7)
    attention.nf4_rope_table(64, 32, scaling=scaling, factor=4.0, high=9.0, out=out, stream=7)
    assert [(c["low"], c["high"]) for c in calls] == [(1.0, high), (1.0, 9.0)]


def test_rope_table_goes_to_the_device_of_its_output(attention, calls, monkeypatch):
    out = Table((64, 16, 2), "cuda:1")
    assert attention.nf4_rope_table(64, 32, out=out) is out
    attention.nf4_rope_table(64, 32, out=out, stream=7)
    assert [(c["stream"], c["device"]) for c in calls] == [(101, 1), (7, 1)]
    assert not hasattr(out, "kept_for")  # a given output is the caller's to keep
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: Table(shape, device))
    made = attention.nf4_rope_table(64, 32, device="cuda:1", stream=7)
    assert (calls[-1]["stream"], calls[-1]["device"]) == (7, 1)
    assert (made.kept_for.cuda_stream, made.kept_for.device) == (7, torch.device("cuda:1"))
    assert attention.nf4_rope_table(64, 32, device="cuda:1", stream=0).kept_for.cuda_stream == 0
    assert not hasattr(attention.nf4_rope_table(64, 32, device="cuda:1"), "kept_for")


def test_the_rest_of_the_package_without_the_compiled_half(attention, tmp_path):
    """Without _attention.so, or with one that does not load, the other entry points are as they were, and the calls of
    the attention side say what is missing."""
    package = os.path.dirname(attention.__file__)
    copy = tmp_path / os.path.basename(package)
    shutil.copytree(package, copy, ignore=shutil.ignore_patterns("_build", "csrc", "__pycache__", "_attention.so"))
    code = """if True:
        from w4a16_gemv_gb300 import *
        import w4a16_gemv_gb300 as nf4
        assert nf4.__file__.startswith({here!r}), nf4.__file__
        assert nf4_version() > 0 and nf4_status_string(0) and nf4.DecodeStep and nf4_gemv and nf4_dequant
        for call in (nf4_rope_table, nf4_qk_norm_rope, nf4_kv_append, nf4_prefix_attention,
                     nf4_prefix_attention_workspace_size):
            try:
                call(1, 2)
            except ImportError as e:
                assert call.__name__ in str(e) and "_attention" in str(e), e
            else:
                raise AssertionError(call)
        """.format(here=str(tmp_path))
    for content in (None, b"not a shared object"):
        if content is not None:
            (copy / "_attention.so").write_bytes(content)
        p = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
        assert p.returncode == 0, p.stderr


def test_another_torch_or_interpreter_asks_for_a_build(monkeypatch):
    import __graft_entry__
    b = __graft_entry__._build_module()
    b.build()
    assert not b._stale()
    key = b._binding_key()
    monkeypatch.setattr(b, "_binding_key", lambda: key + "1")
    assert b._stale()

"""Attention side of the libnf4 binding (``include/nf4_attention.h``): rotary tables, the norm and
rotation of queries and keys, the append to a paged cache and attention over a shared prefix.

As in the rest of the binding: tensors are checked for device, dtype, shape and a contiguous last
dimension (other strides are free), and their pointers go to the C ABI with the current stream.
A paged cache is a pair of tensors [pages, page_size, kv_heads, head_dim]; a cache stored as
[pages, kv_heads, page_size, head_dim] is passed as its ``transpose(1, 2)`` view. The calls made
for every layer of a token are compiled (``csrc/attention_binding.cpp``).
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import NF4Error, _check, _lib, _stream

_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_attention.so")
if not os.path.exists(_PATH):
    raise ImportError(f"{_PATH} is not built: run `python -c \"import __graft_entry__ as g; g.build()\"`")

from . import _attention  # noqa: E402
from ._attention import (nf4_kv_append, nf4_prefix_attention,  # noqa: E402
                         nf4_prefix_attention_workspace_size, nf4_qk_norm_rope)

__all__ = ["nf4_rope_table", "nf4_qk_norm_rope", "nf4_kv_append", "nf4_prefix_attention",
           "nf4_prefix_attention_workspace_size"]

_attention._set_errors(NF4Error, torch.OutOfMemoryError)


class _RopeTableArgs(ctypes.Structure):
    """nf4_rope_table_args of include/nf4_attention.h."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_int64), ("rot_dim", ctypes.c_int64),
                ("scaling", ctypes.c_int64), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("original_positions", ctypes.c_double),
                ("magnitude", ctypes.c_double)]


_lib.nf4_rope_table.argtypes = [ctypes.POINTER(_RopeTableArgs), ctypes.c_void_p]
_lib.nf4_rope_table.restype = ctypes.c_int

_SCALINGS = {"plain": 0, "linear": 1, "bands": 2, "ramp": 3}
_HIGH = {"ramp": 32.0}  # default of `high` (4 for the others), as published


def nf4_rope_table(positions: int, rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                   low: float = 1.0, high: float | None = None, original_positions: float = 8192.0, magnitude: float = 1.0,
                   out: torch.Tensor | None = None, device=None, stream=None) -> torch.Tensor:
    """(cos, sin) of every position's angles, float32 [positions, rot_dim / 2, 2]; ``scaling`` is plain, linear,
    bands (by wavelength) or ramp (by index), with the parameters of nf4_rope_scaling. ``high`` defaults to 4 for
    bands and to 32 for ramp."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    shape = (max(positions, 0), max(rot_dim, 0) // 2, 2)
    fresh = out is None
    if fresh:
        out = torch.empty(shape, dtype=torch.float32, device=device or "cuda")
    if out.dtype != torch.float32:
        raise TypeError(f"out must be torch.float32, got {out.dtype}")
    if not out.is_cuda or out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous CUDA tensor of shape {shape}")
    args = _RopeTableArgs(out.data_ptr(), positions, rot_dim, _SCALINGS[scaling], base, factor, low,
                          _HIGH.get(scaling, 4.0) if high is None else high, original_positions, magnitude)
    with torch.cuda.device(out.device):  # its stream is the default, and the launch goes to the current device
        handle = _stream(stream)
        if fresh and stream is not None and out.numel() > 0:  # kept from reuse until that stream is done with it
            out.record_stream(torch.cuda.ExternalStream(handle, device=out.device) if handle
                              else torch.cuda.default_stream(out.device))
        _check(_lib.nf4_rope_table(ctypes.byref(args), handle), "nf4_rope_table")
    return out

"""Attention side of the libnf4 binding (``include/nf4_attention.h``): rotary tables, the norm and
rotation of queries and keys, the append to a paged cache and attention over a shared prefix.

As in the rest of the binding: tensors are checked for device, dtype, shape and a contiguous last
dimension (other strides are free), and their pointers go to the C ABI with the current stream.
A paged cache is a pair of tensors [pages, page_size, kv_heads, head_dim]; a cache stored as
[pages, kv_heads, page_size, head_dim] is passed as its ``transpose(1, 2)`` view.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import NF4_BF16, NF4_F32, NF4_FP16, _check, _lib, _stream

__all__ = ["nf4_rope_table", "nf4_qk_norm_rope", "nf4_kv_append", "nf4_prefix_attention",
           "nf4_prefix_attention_workspace_size"]

_lib.nf4_rope_table.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
_lib.nf4_rope_table.restype = ctypes.c_int
_lib.nf4_qk_norm_rope.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
_lib.nf4_qk_norm_rope.restype = ctypes.c_int
_lib.nf4_kv_append.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
_lib.nf4_kv_append.restype = ctypes.c_int
_lib.nf4_prefix_attention.argtypes = [ctypes.c_char_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
_lib.nf4_prefix_attention.restype = ctypes.c_int
_lib.nf4_prefix_attention_workspace_size.argtypes = [ctypes.c_char_p]
_lib.nf4_prefix_attention_workspace_size.restype = ctypes.c_size_t

# The argument structures: 8-byte fields in the order of the header (q: integer or pointer, d: double).
_TABLE = struct.Struct("=4q6d")
_QK = struct.Struct("=21qd3q")
_APPEND = struct.Struct("=21qd3q14q")
_ATTN = struct.Struct("=30qd")

_TYPES = {torch.bfloat16: NF4_BF16, torch.float16: NF4_FP16, torch.float32: NF4_F32}
_SCALINGS = {"plain": 0, "linear": 1, "bands": 2, "ramp": 3}


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(t: torch.Tensor, stream) -> int:
    """The stream argument as a handle; None is the current stream of the tensor's device."""
    if stream is None and _current_raw_stream is not None and t.is_cuda:
        return _current_raw_stream(t.get_device())
    return _stream(stream)


# These calls stand between two launches of a decode step, where a microsecond on the host counts: each makes its
# checks as one plain expression per tensor and builds the message only when one fails.

def _bad(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple):
    """Raises what is wrong with a tensor that should be on the GPU, of this dtype and shape."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} must be contiguous" + (" in its last dimension" if len(shape) > 1 else ""))


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> tuple:
    """(pointer, strides of the leading dimensions) of a tensor whose last dimension is contiguous."""
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or (st[-1] != 1 and shape[-1] > 1):
        _bad(t, name, dtype, shape)
    return t.data_ptr(), *st[:-1]


def _flat(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> int:
    """Pointer of a contiguous tensor."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _bad(t, name, dtype, shape)
    return t.data_ptr()


def nf4_rope_table(positions: int, rot_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                   low: float = 1.0, high: float = 4.0, original_positions: float = 8192.0, magnitude: float = 1.0,
                   out: torch.Tensor | None = None, device=None, stream=None) -> torch.Tensor:
    """(cos, sin) of every position's angles, float32 [positions, rot_dim / 2, 2]; ``scaling`` is plain, linear,
    bands (by wavelength) or ramp (by index), with the parameters of nf4_rope_scaling."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}")
    if out is None:
        out = torch.empty((max(positions, 0), max(rot_dim, 0) // 2, 2), dtype=torch.float32, device=device or "cuda")
    ptr = _flat(out, "out", torch.float32, (positions, rot_dim // 2, 2))
    _check(_lib.nf4_rope_table(_TABLE.pack(ptr, positions, rot_dim, _SCALINGS[scaling], base, factor, low, high,
                                           original_positions, magnitude), _stream(stream)), "nf4_rope_table")
    return out


_NO_ROWS = (0, 0, 0, 0, 0, 0, 0)


def _new_rows(x: torch.Tensor, shape: tuple) -> tuple:
    """A new contiguous tensor like x, and its pointer and strides."""
    y = x.new_empty(shape)
    return y, (y.data_ptr(), shape[1] * shape[2], shape[2])


def _qk_fields(q, q_out, k, k_out, append, positions, cos_sin, q_weight, k_weight, eps, interleaved) -> tuple:
    """(q_out, k_out, fields of nf4_qk_norm_rope_args); outputs that are None are made, but no k_out to append."""
    kshape = k.shape
    tokens, k_heads, dim = kshape
    dt = k.dtype
    code = _TYPES.get(dt)
    if code is None:
        raise TypeError("q and k must be bf16, fp16 or fp32")
    tshape = cos_sin.shape
    if len(tshape) != 3 or tshape[2] != 2:
        raise ValueError("cos_sin must have shape [positions, rot_dim / 2, 2]")
    qf = _NO_ROWS
    if q is not None:
        heads = q.shape[1]
        shape = (tokens, heads, dim)
        rows = _rows(q, "q", dt, shape)
        if q_out is None:
            q_out, orows = _new_rows(q, shape)
        else:
            orows = _rows(q_out, "q_out", dt, shape)
        qf = (*rows, *orows, heads)
    krows = _rows(k, "k", dt, kshape)
    if append:
        orows = (0, 0, 0)
    elif k_out is None:
        k_out, orows = _new_rows(k, kshape)
    else:
        orows = _rows(k_out, "k_out", dt, kshape)
    return q_out, k_out, (*qf, *krows, *orows, k_heads, _flat(positions, "positions", torch.int64, (tokens,)),
                          _flat(cos_sin, "cos_sin", torch.float32, tshape), tshape[0], 2 * tshape[1],
                          1 if interleaved else 0,
                          _flat(q_weight, "q_weight", dt, (dim,)) if q_weight is not None else 0,
                          _flat(k_weight, "k_weight", dt, (dim,)) if k_weight is not None else 0,
                          eps, tokens, dim, code)


def nf4_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                     interleaved: bool = False, q_out: torch.Tensor | None = None,
                     k_out: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Norm (where a weight is given) and rotation of q [tokens, q_heads, dim] and k [tokens, k_heads, dim];
    positions int64 [tokens], cos_sin as from nf4_rope_table. Returns (q_out, k_out), new tensors unless given
    (an output may be its input)."""
    q_out, k_out, f = _qk_fields(q, q_out, k, k_out, False, positions, cos_sin, q_weight, k_weight, eps, interleaved)
    status = _lib.nf4_qk_norm_rope(_QK.pack(*f), _stream_of(q, stream))
    if status:
        _check(status, "nf4_qk_norm_rope")
    return q_out, k_out


def nf4_kv_append(k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor, k: torch.Tensor,
                  v: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor, q: torch.Tensor | None = None,
                  q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                  interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Writes the normed and rotated k and the v of each token to slot ``slots[token]`` (int64, page * page_size +
    offset; negative: nowhere) of the paged caches [pages, page_size, kv_heads, dim]. With q, its rows are normed
    and rotated in the same launch and returned."""
    kshape = k.shape
    dt = k.dtype
    pages, page_size = k_cache.shape[:2]
    shape = (pages, page_size, kshape[1], kshape[2])
    q_out, _, f = _qk_fields(q, q_out, k, None, True, positions, cos_sin, q_weight, k_weight, eps, interleaved)
    args = _APPEND.pack(*f, *_rows(v, "v", dt, kshape), _flat(slots, "slots", torch.int64, (kshape[0],)),
                        *_rows(k_cache, "k_cache", dt, shape), *_rows(v_cache, "v_cache", dt, shape), pages, page_size)
    status = _lib.nf4_kv_append(args, _stream_of(k, stream))
    if status:
        _check(status, "nf4_kv_append")
    return q_out


def _attention_args(q, out_rows, lse, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens, cu_q,
                    scale):
    qshape = q.shape
    tokens, heads, dim = qshape
    dt = q.dtype
    code = _TYPES.get(dt)
    if code is None:
        raise TypeError("q must be bf16 or fp16")
    shape = k_cache.shape
    pages, page_size, k_heads, kdim = shape
    if kdim != dim:
        raise ValueError(f"k_cache has head_dim {kdim}, q has {dim}")
    sshape = suffix_pages.shape
    batch, width = sshape
    pshape = prefix_pages.shape
    if len(pshape) != 1 or pshape[0] * page_size < prefix_len:
        raise ValueError(f"prefix_pages of shape {tuple(pshape)}, pages of {page_size}, prefix_len {prefix_len}")
    return _ATTN.pack(*_rows(q, "q", dt, qshape), *out_rows,
                      0 if lse is None else _flat(lse, "lse", torch.float32, (tokens, heads)),
                      *_rows(k_cache, "k_cache", dt, shape), *_rows(v_cache, "v_cache", dt, shape), pages, page_size,
                      _flat(prefix_pages, "prefix_pages", torch.int32, pshape), prefix_len,
                      *_rows(suffix_pages, "suffix_pages", torch.int32, sshape), width,
                      _flat(suffix_lens, "suffix_lens", torch.int32, (batch,)),
                      0 if cu_q is None else _flat(cu_q, "cu_q", torch.int32, (batch + 1,)),
                      batch, tokens, heads, k_heads, dim, code, scale)


def nf4_prefix_attention_workspace_size(q, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens,
                                        cu_q=None, scale: float = 1.0) -> int:
    """Bytes of workspace that nf4_prefix_attention needs for tensors of these shapes."""
    return int(_lib.nf4_prefix_attention_workspace_size(
        _attention_args(q, (0, 0, 0), None, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens, cu_q, scale)))


def nf4_prefix_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, prefix_pages: torch.Tensor,
                         prefix_len: int, suffix_pages: torch.Tensor, suffix_lens: torch.Tensor,
                         cu_q: torch.Tensor | None = None, scale: float | None = None,
                         out: torch.Tensor | None = None, return_lse: bool = False,
                         lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of q [tokens, q_heads, dim] over a paged cache [pages, page_size, kv_heads, dim]: the
    ``prefix_len`` keys on ``prefix_pages`` (int32) that the whole batch shares, then each sequence's own
    ``suffix_lens`` (int32 [batch]) keys on its row of ``suffix_pages`` (int32 [batch, width]), causal among the
    sequence's tokens cu_q[b] .. cu_q[b + 1] - 1 (int32 [batch + 1]; None: one token each). Returns out, or
    (out, lse) with ``return_lse``. The scale defaults to 1 / sqrt(dim)."""
    shape = q.shape
    if out is None:
        out, out_rows = _new_rows(q, shape)
    else:
        out_rows = _rows(out, "out", q.dtype, shape)
    if return_lse and lse is None:
        lse = q.new_empty(shape[:2], dtype=torch.float32)
    if scale is None:
        scale = shape[2] ** -0.5
    s = _stream_of(q, stream)
    args = _attention_args(q, out_rows, lse, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens,
                           cu_q, scale)
    if workspace is not None:
        ws, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        if not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
    else:
        ws, size = None, _lib.nf4_prefix_attention_workspace_size(args)
        if size > 0:
            workspace = q.new_empty(size, dtype=torch.uint8)
            ws = workspace.data_ptr()
            if stream is not None:  # the allocator may not hand it out again before this stream is done with it
                workspace.record_stream(stream if isinstance(stream, torch.cuda.Stream)
                                        else torch.cuda.ExternalStream(s))
    status = _lib.nf4_prefix_attention(args, ws, size, s)
    if status:
        _check(status, "nf4_prefix_attention")
    return (out, lse) if return_lse else out

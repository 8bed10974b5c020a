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


def _view(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple) -> int:
    """Pointer of a CUDA tensor of the given dtype and shape whose last dimension is contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
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
    ptr = _view(out, "out", torch.float32, (positions, rot_dim // 2, 2))
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    _check(_lib.nf4_rope_table(_TABLE.pack(ptr, positions, rot_dim, _SCALINGS[scaling], base, factor, low, high,
                                           original_positions, magnitude), _stream(stream)), "nf4_rope_table")
    return out


def _qk_fields(q, q_out, k, k_out, positions, cos_sin, q_weight, k_weight, eps, interleaved) -> tuple:
    """The fields of nf4_qk_norm_rope_args; q, or k_out, may be None."""
    tokens, k_heads, dim = k.shape
    dt = k.dtype
    if dt not in _TYPES:
        raise TypeError("q and k must be bf16, fp16 or fp32")
    if cos_sin.dim() != 3 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be contiguous, of shape [positions, rot_dim / 2, 2]")
    max_pos, half, _ = cos_sin.shape
    if not positions.is_contiguous():
        raise ValueError("positions must be contiguous")
    pos = _view(positions, "positions", torch.int64, (tokens,))
    table = _view(cos_sin, "cos_sin", torch.float32, (max_pos, half, 2))
    kp = _view(k, "k", dt, k.shape)
    if q is not None:
        heads = q.shape[1]
        shape = (tokens, heads, dim)
        qs, qos = q.stride(), q_out.stride()
        qf = (_view(q, "q", dt, shape), qs[0], qs[1], _view(q_out, "q_out", dt, shape), qos[0], qos[1], heads)
    else:
        qf = (0, 0, 0, 0, 0, 0, 0)
    ks = k.stride()
    if k_out is not None:
        kos = k_out.stride()
        kf = (kp, ks[0], ks[1], _view(k_out, "k_out", dt, k.shape), kos[0], kos[1], k_heads)
    else:
        kf = (kp, ks[0], ks[1], 0, 0, 0, k_heads)
    return (*qf, *kf, pos, table, max_pos, 2 * half, 1 if interleaved else 0,
            _view(q_weight, "q_weight", dt, (dim,)) if q_weight is not None else 0,
            _view(k_weight, "k_weight", dt, (dim,)) if k_weight is not None else 0,
            eps, tokens, dim, _TYPES[dt])


def nf4_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor,
                     q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                     interleaved: bool = False, q_out: torch.Tensor | None = None,
                     k_out: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Norm (where a weight is given) and rotation of q [tokens, q_heads, dim] and k [tokens, k_heads, dim];
    positions int64 [tokens], cos_sin as from nf4_rope_table. Returns (q_out, k_out), new tensors unless given
    (an output may be its input)."""
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    args = _QK.pack(*_qk_fields(q, q_out, k, k_out, positions, cos_sin, q_weight, k_weight, eps, interleaved))
    _check(_lib.nf4_qk_norm_rope(args, _stream(stream)), "nf4_qk_norm_rope")
    return q_out, k_out


def nf4_kv_append(k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor, k: torch.Tensor,
                  v: torch.Tensor, positions: torch.Tensor, cos_sin: torch.Tensor, q: torch.Tensor | None = None,
                  q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                  interleaved: bool = False, q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Writes the normed and rotated k and the v of each token to slot ``slots[token]`` (int64, page * page_size +
    offset; negative: nowhere) of the paged caches [pages, page_size, kv_heads, dim]. With q, its rows are normed
    and rotated in the same launch and returned."""
    tokens, heads, dim = k.shape
    dt = k.dtype
    pages, page_size = k_cache.shape[0], k_cache.shape[1]
    shape = (pages, page_size, heads, dim)
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if not slots.is_contiguous():
        raise ValueError("slots must be contiguous")
    vs, kc, vc = v.stride(), k_cache.stride(), v_cache.stride()
    args = _APPEND.pack(*_qk_fields(q, q_out, k, None, positions, cos_sin, q_weight, k_weight, eps, interleaved),
                        _view(v, "v", dt, k.shape), vs[0], vs[1], _view(slots, "slots", torch.int64, (tokens,)),
                        _view(k_cache, "k_cache", dt, shape), kc[0], kc[1], kc[2],
                        _view(v_cache, "v_cache", dt, shape), vc[0], vc[1], vc[2], pages, page_size)
    _check(_lib.nf4_kv_append(args, _stream(stream)), "nf4_kv_append")
    return q_out


def _attention_args(q, out, lse, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens, cu_q, scale):
    tokens, heads, dim = q.shape
    dt = q.dtype
    if dt not in _TYPES:
        raise TypeError("q must be bf16 or fp16")
    shape = k_cache.shape
    pages, page_size, k_heads, _ = shape
    if shape[3] != dim:
        raise ValueError(f"k_cache has head_dim {shape[3]}, q has {dim}")
    batch, width = suffix_pages.shape
    if prefix_pages.dim() != 1 or not prefix_pages.is_contiguous():
        raise ValueError("prefix_pages must be contiguous, of one dimension")
    if prefix_pages.shape[0] * page_size < prefix_len:
        raise ValueError(f"prefix_pages has {prefix_pages.shape[0]} pages of {page_size}, prefix_len is {prefix_len}")
    if not suffix_lens.is_contiguous() or (cu_q is not None and not cu_q.is_contiguous()):
        raise ValueError("suffix_lens and cu_q must be contiguous")
    qs, os, kc, vc = q.stride(), out.stride(), k_cache.stride(), v_cache.stride()
    return _ATTN.pack(_view(q, "q", dt, q.shape), qs[0], qs[1], _view(out, "out", dt, q.shape), os[0], os[1],
                      0 if lse is None else _view(lse, "lse", torch.float32, (tokens, heads)),
                      _view(k_cache, "k_cache", dt, shape), kc[0], kc[1], kc[2],
                      _view(v_cache, "v_cache", dt, shape), vc[0], vc[1], vc[2], pages, page_size,
                      _view(prefix_pages, "prefix_pages", torch.int32, prefix_pages.shape), prefix_len,
                      _view(suffix_pages, "suffix_pages", torch.int32, (batch, width)), suffix_pages.stride(0), width,
                      _view(suffix_lens, "suffix_lens", torch.int32, (batch,)),
                      0 if cu_q is None else _view(cu_q, "cu_q", torch.int32, (batch + 1,)),
                      batch, tokens, heads, k_heads, dim, _TYPES[dt], scale)


def nf4_prefix_attention_workspace_size(q, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens,
                                        cu_q=None, scale: float = 1.0) -> int:
    """Bytes of workspace that nf4_prefix_attention needs for tensors of these shapes."""
    return int(_lib.nf4_prefix_attention_workspace_size(
        _attention_args(q, q, None, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens, cu_q, scale)))


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
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    if lse is not None and not lse.is_contiguous():
        raise ValueError("lse must be contiguous")
    if scale is None:
        scale = q.shape[2] ** -0.5
    s = _stream(stream)
    args = _attention_args(q, out, lse, k_cache, v_cache, prefix_pages, prefix_len, suffix_pages, suffix_lens, cu_q,
                           scale)
    need = _lib.nf4_prefix_attention_workspace_size(args)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        if stream is not None:  # the allocator may not hand it out again before this stream is done with it
            workspace.record_stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(s))
    _check(_lib.nf4_prefix_attention(args, workspace.data_ptr() if workspace is not None else None,
                                     workspace.numel() * workspace.element_size() if workspace is not None else 0, s),
           "nf4_prefix_attention")
    return (out, lse) if return_lse else out

"""A decode step around its GEMVs (``include/nf4_decoding.h``): page tables and slots from the requests'
lengths, attention for trees of drafted tokens, adjusted logits and their best tokens, and taking the
accepted branch of a tree into the paged cache.

The conventions are the attention side's (``attention.py``): tensors are checked for device, dtype, shape
and a contiguous last dimension, and their pointers go to the C ABI with the current stream. All calls are
compiled (``csrc/decoding_binding.cpp``); none synchronises, so that a step of them can be recorded into a
CUDA graph and replayed. int32 tensors are given and returned; sequences are ragged, by ``cu_q`` offsets.
"""
from __future__ import annotations

from . import attention  # noqa: F401  (loads the compiled half, and says what is missing without it)
from ._attention import (nf4_adjust_logits, nf4_kv_pages, nf4_tree_attention,
                         nf4_tree_attention_workspace_size, nf4_tree_commit)

__all__ = ["nf4_kv_pages", "nf4_tree_attention", "nf4_tree_attention_workspace_size", "nf4_adjust_logits",
           "nf4_tree_commit"]

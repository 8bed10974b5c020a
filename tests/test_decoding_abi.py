"""The C ABI of include/nf4_decoding.h without a GPU: exports, the layout of the argument structures,
and the refusals on the host before any CUDA call; and what the Python side refuses."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nf4_decoding.h")

OK, ERR_NULL, ERR_SIZE, ERR_BS, ERR_ALIGN, ERR_DTYPE, ERR_BATCH, ERR_CUDA, ERR_WS = range(9)
BF16, FP16, F32 = 0, 1, 2
A = 0x100000  # a fake, well-aligned address: never dereferenced by these calls
B = 0x200000

ATTENTION = ("q q_token_stride q_head_stride out out_token_stride out_head_stride lse k_cache k_page_stride k_slot_stride "
             "k_head_stride v_cache v_page_stride v_slot_stride v_head_stride num_pages page_size prefix_pages prefix_len "
             "suffix_pages suffix_pages_stride suffix_pages_width suffix_lens cu_q batch tokens q_heads k_heads head_dim "
             "dtype scale").split()
FIELDS = {
    "nf4_kv_pages_args":
        "lens cu_q depths page_table page_table_stride width held free_pages capacity free_count slots positions "
        "new_lens new_held new_free_count batch tokens page_size first_position",
    "nf4_tree_attention_args": " ".join(ATTENTION) + " tree_mask tree_mask_stride tree_words",
    "nf4_adjust_logits_args":
        "logits logits_stride out out_stride best rows vocab dtype requests cu_rows history history_stride "
        "history_width history_lens prompt_lens repetition frequency presence bias_tokens bias_values bias_stride "
        "bias_width mask mask_stride mask_count mask_rows draft_tokens tree_mask tree_mask_stride tree_words",
    "nf4_tree_commit_args":
        "parents draft_tokens targets cu_q lens batch tokens max_path accepted path chosen new_lens k_cache "
        "k_layer_stride k_page_stride k_slot_stride k_head_stride v_cache v_layer_stride v_page_stride v_slot_stride "
        "v_head_stride layers num_pages page_size k_heads head_dim page_table page_table_stride width",
}
STRUCTS = {name: type(name, (ctypes.Structure,), {"_fields_": [
    (f, ctypes.c_double if f == "scale" else ctypes.c_int64) for f in fields.split()]}) for name, fields in FIELDS.items()}

GOOD = {
    "nf4_kv_pages_args":
        dict(lens=A, cu_q=A, depths=A, page_table=A, page_table_stride=9, width=9, held=A, free_pages=A, capacity=50,
             free_count=A, slots=A, positions=A, new_lens=B, new_held=A, new_free_count=A, batch=3, tokens=5, page_size=16,
             first_position=7),
    "nf4_tree_attention_args":
        dict(q=A, q_token_stride=512, q_head_stride=128, out=A, out_token_stride=512, out_head_stride=128, lse=A,
             k_cache=A, k_page_stride=4096, k_slot_stride=256, k_head_stride=128, v_cache=A, v_page_stride=4096,
             v_slot_stride=256, v_head_stride=128, num_pages=50, page_size=16, prefix_pages=A, prefix_len=100,
             suffix_pages=A, suffix_pages_stride=4, suffix_pages_width=4, suffix_lens=A, cu_q=A, batch=3, tokens=5,
             q_heads=4, k_heads=2, head_dim=128, dtype=BF16, scale=0.1, tree_mask=A, tree_mask_stride=1, tree_words=1),
    "nf4_adjust_logits_args":
        dict(logits=A, logits_stride=1000, out=A, out_stride=1000, best=A, rows=5, vocab=1000, dtype=F32, requests=3,
             cu_rows=A, history=A, history_stride=64, history_width=64, history_lens=A, prompt_lens=A, repetition=A,
             frequency=A, presence=A, bias_tokens=A, bias_values=A, bias_stride=8, bias_width=8, mask=A, mask_stride=32,
             mask_count=5, mask_rows=A, draft_tokens=A, tree_mask=A, tree_mask_stride=1, tree_words=1),
    "nf4_tree_commit_args":
        dict(parents=A, draft_tokens=A, targets=A, cu_q=A, lens=A, batch=3, tokens=5, max_path=8, accepted=A, path=A,
             chosen=A, new_lens=B, k_cache=A + 4096, k_layer_stride=65536, k_page_stride=4096, k_slot_stride=256,
             k_head_stride=128, v_cache=A, v_layer_stride=65536, v_page_stride=4096, v_slot_stride=256, v_head_stride=128,
             layers=2, num_pages=50, page_size=16, k_heads=2, head_dim=128, page_table=A, page_table_stride=4, width=4),
}


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    lib = ctypes.CDLL(__graft_entry__._build_module().build())
    for name in ("nf4_kv_pages", "nf4_adjust_logits", "nf4_tree_commit"):
        getattr(lib, name).argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.nf4_tree_attention.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.nf4_tree_attention_workspace_size.argtypes = [ctypes.c_void_p]
    lib.nf4_tree_attention_workspace_size.restype = ctypes.c_size_t
    return lib


def call(lib, name, ws=A, **kw):
    args = STRUCTS[name + "_args"](**{**GOOD[name + "_args"], **kw})
    rest = (ws or None, 1 << 30, None) if name == "nf4_tree_attention" else (None,)
    return getattr(lib, name)(ctypes.byref(args), *rest)


def test_exports_every_declared_symbol(lib):
    names = re.findall(r"NF4_API\s+[\w\s\*]+?\b(nf4_\w+)\s*\(", open(HEADER).read())
    assert set(names) == {"nf4_kv_pages", "nf4_tree_attention", "nf4_tree_attention_workspace_size", "nf4_adjust_logits",
                          "nf4_tree_commit"}
    import w4a16_gemv_gb300 as nf4
    import w4a16_gemv_gb300.decoding as decoding
    for n in names:
        assert hasattr(lib, n) and n in nf4.__all__ and getattr(nf4, n) is getattr(decoding, n), n


def test_structures_are_eight_byte_fields(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    body = ""
    for name, fields in FIELDS.items():
        for f in fields.split():
            nested = "attention." if name == "nf4_tree_attention_args" and f in ATTENTION else ""
            body += f'printf("%zu ", offsetof({name}, {nested}{f}));'
        body += f'printf("%zu\\n", sizeof({name}));'
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "nf4_decoding.h"\n'
                   f"int main(void) {{ {body} return 0; }}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    for (name, fields), line in zip(FIELDS.items(), lines):
        assert [int(v) for v in line.split()] == list(range(0, 8 * len(fields.split()) + 1, 8)), name
        assert ctypes.sizeof(STRUCTS[name]) == 8 * len(fields.split())


def test_null_argument_structures(lib):
    for name in ("nf4_kv_pages", "nf4_adjust_logits", "nf4_tree_commit"):
        assert getattr(lib, name)(None, None) == ERR_NULL
    assert lib.nf4_tree_attention(None, None, 0, None) == ERR_NULL
    assert lib.nf4_tree_attention_workspace_size(None) == 0


@pytest.mark.parametrize("name,status,cases", [
    ("nf4_kv_pages", ERR_SIZE,
     [dict(batch=-1), dict(batch=(1 << 20) + 1), dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(page_size=0),
      dict(page_size=65537), dict(width=-1), dict(width=(1 << 26) + 1, page_table_stride=1 << 30), dict(capacity=-1),
      dict(capacity=1 << 31), dict(first_position=-1), dict(first_position=(1 << 30) + 1), dict(page_table_stride=8),
      dict(page_table_stride=-1), dict(cu_q=0), dict(new_lens=A)]),
    ("nf4_kv_pages", ERR_NULL,
     [dict(lens=0), dict(held=0), dict(new_lens=0), dict(new_held=0), dict(page_table=0), dict(free_pages=0),
      dict(free_count=0), dict(new_free_count=0), dict(slots=0)]),
    ("nf4_kv_pages", ERR_ALIGN,
     [dict(lens=A + 2), dict(cu_q=A + 1), dict(depths=A + 2), dict(page_table=A + 2), dict(held=A + 2), dict(slots=A + 4),
      dict(positions=A + 4), dict(free_pages=A + 2), dict(free_count=A + 2), dict(new_free_count=A + 1)]),
    ("nf4_tree_attention", ERR_SIZE,
     [dict(tree_words=0), dict(tree_words=1025), dict(tree_mask_stride=-1), dict(tokens=-1), dict(head_dim=20),
      dict(scale=0.0), dict(k_heads=3), dict(cu_q=0)]),
    ("nf4_tree_attention", ERR_NULL, [dict(tree_mask=0), dict(q=0), dict(out=0), dict(suffix_pages=0), dict(k_cache=0)]),
    ("nf4_tree_attention", ERR_ALIGN, [dict(tree_mask=A + 4), dict(q=A + 2), dict(q_token_stride=511), dict(cu_q=A + 2)]),
    ("nf4_tree_attention", ERR_DTYPE, [dict(dtype=F32)]),
    ("nf4_tree_attention", ERR_WS, [dict(ws=0), dict(ws=A + 8)]),
    ("nf4_adjust_logits", ERR_SIZE,
     [dict(rows=-1), dict(rows=(1 << 20) + 1), dict(vocab=0), dict(vocab=(1 << 24) + 1, out_stride=1 << 30),
      dict(requests=-1), dict(requests=(1 << 20) + 1), dict(logits_stride=-1), dict(out_stride=999), dict(out_stride=-1),
      dict(history_width=-1), dict(history_width=(1 << 28) + 1), dict(history_stride=-1), dict(bias_width=1025),
      dict(bias_width=-1), dict(bias_stride=-1), dict(mask_count=-1), dict(mask_stride=-1), dict(mask_rows=0, mask_count=4),
      dict(tree_words=0), dict(tree_words=1025), dict(tree_mask_stride=-1), dict(cu_rows=0)]),
    ("nf4_adjust_logits", ERR_DTYPE, [dict(dtype=3), dict(dtype=-1)]),
    ("nf4_adjust_logits", ERR_NULL, [dict(logits=0), dict(out=0), dict(history_lens=0), dict(bias_values=0), dict(tree_mask=0)]),
    ("nf4_adjust_logits", ERR_ALIGN,
     [dict(logits=A + 2), dict(out=A + 2), dict(logits=A + 1, dtype=BF16), dict(best=A + 2), dict(history=A + 2),
      dict(mask=A + 2), dict(tree_mask=A + 4), dict(bias_values=A + 2), dict(repetition=A + 1)]),
    ("nf4_tree_commit", ERR_SIZE,
     [dict(batch=-1), dict(batch=(1 << 20) + 1), dict(tokens=-1), dict(max_path=0), dict(max_path=1025), dict(cu_q=0),
      dict(layers=-1), dict(layers=65536), dict(num_pages=-1), dict(page_size=0), dict(k_heads=0), dict(head_dim=0),
      dict(head_dim=513), dict(width=-1), dict(page_table_stride=-1), dict(k_slot_stride=-1), dict(v_layer_stride=-1),
      dict(k_layer_stride=0), dict(v_layer_stride=0), dict(k_cache=A), dict(new_lens=A)]),
    ("nf4_tree_commit", ERR_NULL,
     [dict(parents=0), dict(draft_tokens=0), dict(targets=0), dict(lens=0), dict(accepted=0), dict(path=0), dict(chosen=0),
      dict(new_lens=0), dict(k_cache=0), dict(v_cache=0), dict(page_table=0)]),
    ("nf4_tree_commit", ERR_ALIGN,
     [dict(parents=A + 2), dict(targets=A + 1), dict(path=A + 2), dict(k_cache=A + 1), dict(v_cache=A + 1)]),
])
def test_refusals(lib, name, status, cases):
    for kw in cases:
        assert call(lib, name, **kw) == status, kw


def test_adjusted_logits_over_other_rows_are_refused(lib):
    """out is logits itself, or shares no element with it."""
    for kw in (dict(out=A + 4), dict(out=A - 4), dict(out=A + 4 * 5000 - 4), dict(out_stride=2000), dict(logits_stride=0),
               dict(out=A + 4 * 1000), dict(rows=1, out=A + 4), dict(vocab=600, out=A + 4 * 500),
               dict(vocab=500, out=A + 4 * 501), dict(vocab=500, out=A + 4 * 499), dict(vocab=400, out=A + 4 * 500, out_stride=1001)):
        assert call(lib, "nf4_adjust_logits", **kw) == ERR_SIZE, kw


def test_caches_whose_rows_are_at_two_indices_are_refused(lib):
    """A stride of 0 of a dimension of more than one; of one element it is not used."""
    for cache in "kv":
        for dim, one in (("layer", "layers"), ("page", "num_pages"), ("slot", "page_size"), ("head", "k_heads")):
            kw = {f"{cache}_{dim}_stride": 0}
            assert call(lib, "nf4_tree_commit", **kw) == ERR_SIZE, kw
            assert call(lib, "nf4_tree_commit", batch=0, **kw, **{one: 1}) == OK, kw


def test_lengths_written_over_others_are_refused(lib):
    """Lists that are read while they are written: the same one only where the call says so, others apart."""
    for off in (0, 4, -4, 8, -8):  # three entries of four bytes
        assert call(lib, "nf4_kv_pages", new_lens=A + off) == ERR_SIZE
        assert call(lib, "nf4_tree_commit", new_lens=A + off) == ERR_SIZE
        if off:
            assert call(lib, "nf4_kv_pages", new_held=A + off) == ERR_SIZE
            assert call(lib, "nf4_tree_commit", new_lens=A + off, k_cache=0, v_cache=0) == ERR_SIZE


def test_calls_without_work(lib):
    assert call(lib, "nf4_kv_pages", batch=0, tokens=0) == OK
    assert call(lib, "nf4_tree_attention", tokens=0, tree_mask=0) == OK
    assert call(lib, "nf4_adjust_logits", rows=0, logits=0) == OK
    assert call(lib, "nf4_tree_commit", batch=0, tokens=0, parents=0) == OK


def test_workspace_of_a_tree(lib):
    """Two numbers and a row in binary32 for each row and range of keys; nothing where one range writes the output."""
    size = lambda **kw: lib.nf4_tree_attention_workspace_size(ctypes.byref(  # noqa: E731
        STRUCTS["nf4_tree_attention_args"](**{**GOOD["nf4_tree_attention_args"], **kw})))
    for kw in (dict(), dict(prefix_len=0, suffix_pages_width=4000, suffix_pages_stride=4000), dict(batch=1, tokens=200)):
        t = {**GOOD["nf4_tree_attention_args"], **kw}
        row = t["tokens"] * t["q_heads"] * (t["head_dim"] * 4 + 8)
        assert size(**kw) > 0 and size(**kw) % row == 0 and size(**kw) // row <= 304, kw
    assert size(tree_words=0) == size(tokens=0) == size(head_dim=4) == 0
    assert size(prefix_len=0, suffix_pages_width=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="these calls would launch")
def test_valid_calls_without_a_gpu_report_cuda(lib):
    for name in ("nf4_kv_pages", "nf4_tree_attention", "nf4_adjust_logits", "nf4_tree_commit"):
        assert call(lib, name) == ERR_CUDA, name


def test_binding_refuses_before_it_looks_at_a_gpu(lib):
    import w4a16_gemv_gb300 as nf4
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        nf4.nf4_kv_pages(i, i.view(2, 1), i, i, i[:1], 16)
    with pytest.raises(TypeError, match="missing"):
        nf4.nf4_kv_pages(i, i.view(2, 1))
    with pytest.raises(ValueError, match="CUDA"):
        nf4.nf4_adjust_logits(torch.zeros(2, 5))
    with pytest.raises(ValueError, match="shape"):
        nf4.nf4_adjust_logits(torch.zeros(5))
    with pytest.raises(TypeError, match="unexpected"):
        nf4.nf4_adjust_logits(torch.zeros(2, 5), temperature=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        nf4.nf4_tree_commit(i, i, i, None, i, 4)
    with pytest.raises(TypeError, match="tensor"):
        nf4.nf4_tree_attention(1, 2, 3, 4, 5, 6, 7, 8)


@pytest.mark.skipif(torch.cuda.is_available(), reason="these calls would launch")
def test_lengths_in_place_and_side_by_side(lib):
    for off in (0, 12, -12):
        assert call(lib, "nf4_kv_pages", new_held=A + off) == ERR_CUDA
        assert call(lib, "nf4_tree_commit", new_lens=A + off, k_cache=0, v_cache=0) == ERR_CUDA

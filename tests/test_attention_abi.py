"""The C ABI of include/nf4_attention.h without a GPU: exports, the layout of the argument
structures, and the refusals on the host before any CUDA call."""
import ctypes
import os
import re
import shutil
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nf4_attention.h")

OK, ERR_NULL, ERR_SIZE, ERR_BS, ERR_ALIGN, ERR_DTYPE, ERR_BATCH, ERR_CUDA, ERR_WS = range(9)
BF16, FP16, F32 = 0, 1, 2
A = 0x100000  # a fake, well-aligned address: never dereferenced by these calls

FIELDS = {
    "nf4_rope_table_args": "cos_sin positions rot_dim scaling base factor low high original_positions magnitude",
    "nf4_qk_norm_rope_args":
        "q q_token_stride q_head_stride q_out q_out_token_stride q_out_head_stride q_heads k k_token_stride "
        "k_head_stride k_out k_out_token_stride k_out_head_stride k_heads positions cos_sin max_positions rot_dim "
        "interleaved q_weight k_weight eps tokens head_dim dtype",
    "nf4_kv_append_args":
        "qk v v_token_stride v_head_stride slots k_cache k_page_stride k_slot_stride k_head_stride v_cache "
        "v_page_stride v_slot_stride v_cache_head_stride num_pages page_size",
    "nf4_prefix_attention_args":
        "q q_token_stride q_head_stride out out_token_stride out_head_stride lse k_cache k_page_stride "
        "k_slot_stride k_head_stride v_cache v_page_stride v_slot_stride v_head_stride num_pages page_size "
        "prefix_pages prefix_len suffix_pages suffix_pages_stride suffix_pages_width suffix_lens cu_q batch tokens "
        "q_heads k_heads head_dim dtype scale",
}


# The structures as 8-byte fields in the order of FIELDS (q: integer or pointer, d: double).
TABLE, QK_ARGS, APPEND, ATTN = (struct.Struct(f) for f in ("=4q6d", "=21qd3q", "=21qd3q14q", "=30qd"))


@pytest.fixture(scope="module")
def att():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import w4a16_gemv_gb300.attention as attention
    return attention


class Lib:
    """The C entry points, taking the argument structure as bytes."""

    def __init__(self, path):
        lib = ctypes.CDLL(path)
        for name, args in (("nf4_rope_table", []), ("nf4_qk_norm_rope", []), ("nf4_kv_append", []),
                           ("nf4_prefix_attention", [ctypes.c_void_p, ctypes.c_size_t]),
                           ("nf4_prefix_attention_workspace_size", None)):
            f = getattr(lib, name)
            f.argtypes = [ctypes.c_char_p] + (args + [ctypes.c_void_p] if args is not None else [])
            f.restype = ctypes.c_int if args is not None else ctypes.c_size_t
            setattr(self, name, f)
        self.nf4_last_cuda_error = lib.nf4_last_cuda_error


@pytest.fixture(scope="module")
def lib(att):
    import w4a16_gemv_gb300 as nf4
    return Lib(nf4.LIB_PATH)


def test_exports_every_declared_symbol(att):
    names = re.findall(r"NF4_API\s+[\w\s\*]+?\b(nf4_\w+)\s*\(", open(HEADER).read())
    assert set(names) == {"nf4_rope_table", "nf4_qk_norm_rope", "nf4_kv_append", "nf4_prefix_attention",
                          "nf4_prefix_attention_workspace_size"}
    for n in names:
        assert hasattr(att._lib, n), n
        assert hasattr(att, n), n


def test_structures_are_eight_byte_fields(tmp_path):
    """Every field is eight bytes, in the order of FIELDS."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    body = ""
    for name, fields in FIELDS.items():
        for f in fields.split():
            body += f'printf("%zu ", offsetof({name}, {f}));'
        body += f'printf("%zu\\n", sizeof({name}));'
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "nf4_attention.h"\n'
                   f"int main(void) {{ {body} return 0; }}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()
    packed = (TABLE, QK_ARGS, APPEND, ATTN)
    for (name, fields), line, st in zip(FIELDS.items(), lines, packed):
        got = [int(v) for v in line.split()]
        assert got[-1] == st.size, name
        if name == "nf4_kv_append_args":
            want = [0] + list(range(got[1], st.size, 8))
            assert got[1] == QK_ARGS.size
        else:
            want = list(range(0, st.size, 8))
        assert got[:-1] == want and len(want) == len(fields.split()), name
    # the doubles stand where the formats have a d
    order = FIELDS["nf4_qk_norm_rope_args"].split()
    assert QK_ARGS.format == "=%dqd%dq" % (order.index("eps"), len(order) - order.index("eps") - 1)
    order = FIELDS["nf4_prefix_attention_args"].split()
    assert ATTN.format == "=%dqd" % order.index("scale")


class Args(dict):
    """Fields by name, packed in the header's order."""

    def pack(self, st, *names):
        return st.pack(*(self[f] for n in names for f in FIELDS[n].split() if f != "qk"))


def table(lib, **kw):
    a = Args(cos_sin=A, positions=64, rot_dim=32, scaling=0, base=10000.0, factor=1.0, low=1.0, high=4.0,
             original_positions=8192.0, magnitude=1.0)
    a.update(kw)
    return lib.nf4_rope_table(a.pack(TABLE, "nf4_rope_table_args"), None)


QK = dict(q=A, q_token_stride=256, q_head_stride=64, q_out=A, q_out_token_stride=256, q_out_head_stride=64, q_heads=4,
          k=A, k_token_stride=128, k_head_stride=64, k_out=A, k_out_token_stride=128, k_out_head_stride=64, k_heads=2,
          positions=A, cos_sin=A, max_positions=100, rot_dim=64, interleaved=0, q_weight=A, k_weight=A, eps=1e-6,
          tokens=3, head_dim=64, dtype=BF16)


def qk(lib, **kw):
    return lib.nf4_qk_norm_rope(Args({**QK, **kw}).pack(QK_ARGS, "nf4_qk_norm_rope_args"), None)


def append(lib, **kw):
    a = Args({**QK, **dict(v=A, v_token_stride=128, v_head_stride=64, slots=A, k_cache=A, k_page_stride=2048,
                           k_slot_stride=128, v_cache=A, v_page_stride=2048, v_slot_stride=128, v_cache_head_stride=64,
                           num_pages=9, page_size=16), **kw})
    qk_fields = [a[f] for f in FIELDS["nf4_qk_norm_rope_args"].split()]
    rest = [a[f] for f in FIELDS["nf4_kv_append_args"].split()[1:]]
    return lib.nf4_kv_append(APPEND.pack(*qk_fields, *rest), None)


ATT = dict(q=A, q_token_stride=512, q_head_stride=128, out=A, out_token_stride=512, out_head_stride=128, lse=A,
           k_cache=A, k_page_stride=4096, k_slot_stride=256, k_head_stride=128, v_cache=A, v_page_stride=4096,
           v_slot_stride=256, v_head_stride=128, num_pages=50, page_size=16, prefix_pages=A, prefix_len=100,
           suffix_pages=A, suffix_pages_stride=4, suffix_pages_width=4, suffix_lens=A, cu_q=A, batch=3, tokens=5,
           q_heads=4, k_heads=2, head_dim=128, dtype=BF16, scale=0.1)


def attend(lib, ws=A, ws_bytes=1 << 30, **kw):
    a = Args({**ATT, **kw}).pack(ATTN, "nf4_prefix_attention_args")
    return lib.nf4_prefix_attention(a, ws or None, ws_bytes, None)


def ws_size(lib, **kw):
    return lib.nf4_prefix_attention_workspace_size(Args({**ATT, **kw}).pack(ATTN, "nf4_prefix_attention_args"))


def test_null_argument_structures(lib):
    assert lib.nf4_rope_table(None, None) == ERR_NULL
    assert lib.nf4_qk_norm_rope(None, None) == ERR_NULL
    assert lib.nf4_kv_append(None, None) == ERR_NULL
    assert lib.nf4_prefix_attention(None, None, 0, None) == ERR_NULL
    assert lib.nf4_prefix_attention_workspace_size(None) == 0


def test_rope_table_refusals(lib):
    for kw in (dict(positions=-1), dict(positions=(1 << 30) + 1), dict(rot_dim=0), dict(rot_dim=31), dict(rot_dim=514),
               dict(scaling=-1), dict(scaling=4), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
               dict(magnitude=0.0), dict(magnitude=float("inf")), dict(scaling=1, factor=0.5),
               dict(scaling=1, factor=float("nan")), dict(scaling=2, low=0.0), dict(scaling=2, low=4.0),
               dict(scaling=3, original_positions=0.0), dict(scaling=3, high=float("inf"))):
        assert table(lib, **kw) == ERR_SIZE, kw
    assert table(lib, positions=0, cos_sin=0) == OK
    assert table(lib, cos_sin=0) == ERR_NULL
    assert table(lib, cos_sin=A + 4) == ERR_ALIGN


@pytest.mark.parametrize("call", [qk, append])
def test_norm_and_rotation_refusals(lib, call):
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(head_dim=0), dict(head_dim=513), dict(q_heads=-1),
               dict(q_heads=65536), dict(k_heads=65536), dict(rot_dim=-2), dict(rot_dim=63), dict(rot_dim=66),
               dict(max_positions=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(interleaved=2),
               dict(q_token_stride=-1), dict(q_out_head_stride=-8), dict(k_head_stride=-1),
               dict(q_token_stride=(1 << 40) + 1)):
        assert call(lib, **kw) == ERR_SIZE, kw
    for d in (-1, 3):
        assert call(lib, dtype=d) == ERR_DTYPE
    for kw in (dict(q=0), dict(q_out=0), dict(k=0), dict(positions=0), dict(cos_sin=0)):
        assert call(lib, **kw) == ERR_NULL, kw
    for kw in (dict(q=A + 1), dict(q_out=A + 1), dict(k=A + 1), dict(q_weight=A + 1), dict(k_weight=A + 1),
               dict(positions=A + 4), dict(cos_sin=A + 4)):
        assert call(lib, **kw) == ERR_ALIGN, kw
    assert call(lib, tokens=0, q=0, k=0, positions=0) == OK


def test_norm_and_rotation_own_refusals(lib):
    assert qk(lib, k_out=0) == ERR_NULL
    assert qk(lib, k_out=A + 1) == ERR_ALIGN
    assert qk(lib, k_out_token_stride=-1) == ERR_SIZE
    assert qk(lib, dtype=F32, q=A + 2) == ERR_ALIGN
    assert qk(lib, q_heads=0, k_heads=0, q=0, k=0) == OK


def test_append_own_refusals(lib):
    assert append(lib, k_heads=0) == ERR_SIZE
    assert append(lib, dtype=F32) == ERR_DTYPE
    for kw in (dict(num_pages=-1), dict(page_size=0), dict(page_size=65537), dict(v_token_stride=-1),
               dict(k_page_stride=-1), dict(v_slot_stride=-1), dict(v_cache_head_stride=(1 << 40) + 1)):
        assert append(lib, **kw) == ERR_SIZE, kw
    for kw in (dict(v=0), dict(slots=0), dict(k_cache=0), dict(v_cache=0)):
        assert append(lib, **kw) == ERR_NULL, kw
    for kw in (dict(v=A + 1), dict(slots=A + 4), dict(k_cache=A + 1), dict(v_cache=A + 1)):
        assert append(lib, **kw) == ERR_ALIGN, kw


def test_prefix_attention_refusals(lib):
    for kw in (dict(batch=-1), dict(batch=(1 << 20) + 1), dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(k_heads=0),
               dict(q_heads=0), dict(q_heads=5), dict(head_dim=0), dict(head_dim=12), dict(head_dim=136),
               dict(num_pages=-1), dict(page_size=0), dict(page_size=65537), dict(prefix_len=-1),
               dict(prefix_len=(1 << 30) + 1), dict(suffix_pages_width=-1), dict(suffix_pages_width=(1 << 26) + 1),
               dict(suffix_pages_stride=-1), dict(q_token_stride=-8), dict(k_slot_stride=-8), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(tokens=1 << 24, q_heads=128), dict(cu_q=0)):
        assert attend(lib, **kw) == ERR_SIZE, kw
    for d in (-1, F32, 3):
        assert attend(lib, dtype=d) == ERR_DTYPE
    for kw in (dict(q=0), dict(out=0), dict(prefix_pages=0), dict(suffix_pages=0), dict(suffix_lens=0),
               dict(k_cache=0), dict(v_cache=0)):
        assert attend(lib, **kw) == ERR_NULL, kw
    for kw in (dict(q=A + 8), dict(out=A + 2), dict(k_cache=A + 8), dict(v_cache=A + 8), dict(lse=A + 2),
               dict(prefix_pages=A + 2), dict(suffix_pages=A + 2), dict(suffix_lens=A + 1), dict(cu_q=A + 2),
               dict(q_token_stride=508), dict(out_head_stride=4), dict(k_slot_stride=250), dict(v_page_stride=4097)):
        assert attend(lib, **kw) == ERR_ALIGN, kw
    assert attend(lib, tokens=0, q=0, out=0) == OK


def test_prefix_attention_workspace(lib):
    need = ws_size(lib)
    assert need > 0
    assert attend(lib, ws_bytes=need - 1) == ERR_WS
    assert attend(lib, ws=0) == ERR_WS
    assert attend(lib, ws=A + 8) == ERR_WS
    assert ws_size(lib, tokens=0) == 0
    assert ws_size(lib, head_dim=12) == 0
    assert ws_size(lib, batch=0, prefix_len=0) == 0
    # pointers are not looked at
    assert ws_size(lib, q=0, out=0, k_cache=0, cu_q=0) == need


def test_cuda_failure_is_reported_as_a_status(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for call in (table, qk, append, attend):
        assert call(lib) == ERR_CUDA, call.__name__
        assert lib.nf4_last_cuda_error() != 0

"""What nf4_prefix_attention plans and refuses on the host, without a GPU."""
import ctypes

import pytest

BF16, FP16 = 0, 1
ERR_SIZE = 2
A = 0x100000  # a fake, well-aligned address: never dereferenced by these calls
NAMES = ("q q_token_stride q_head_stride out out_token_stride out_head_stride lse k_cache k_page_stride k_slot_stride "
         "k_head_stride v_cache v_page_stride v_slot_stride v_head_stride num_pages page_size prefix_pages prefix_len "
         "suffix_pages suffix_pages_stride suffix_pages_width suffix_lens cu_q batch tokens q_heads k_heads head_dim "
         "dtype").split()


class Args(ctypes.Structure):
    """nf4_prefix_attention_args of include/nf4_attention.h."""
    _fields_ = [(n, ctypes.c_int64) for n in NAMES] + [("scale", ctypes.c_double)]


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    path = __graft_entry__._build_module().build()
    lib = ctypes.CDLL(path)
    lib.nf4_prefix_attention.argtypes = [ctypes.POINTER(Args), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.nf4_prefix_attention_workspace_size.argtypes = [ctypes.POINTER(Args)]
    lib.nf4_prefix_attention_workspace_size.restype = ctypes.c_size_t
    return lib


def args(**kw):
    heads, dim = kw.get("q_heads", 4), kw.get("head_dim", 128)
    a = dict.fromkeys(NAMES, A)
    a.update(q_token_stride=heads * dim, q_head_stride=dim, out_token_stride=heads * dim, out_head_stride=dim,
             k_page_stride=4096, k_slot_stride=256, k_head_stride=128, v_page_stride=4096, v_slot_stride=256,
             v_head_stride=128, num_pages=50, page_size=16, prefix_len=100, suffix_pages_stride=4,
             suffix_pages_width=4, batch=3, tokens=5, q_heads=4, k_heads=2, head_dim=128, dtype=BF16, scale=0.1)
    a.update(kw)
    return Args(**a)


@pytest.mark.parametrize("kw,rows", [
    (dict(tokens=608, q_heads=64, batch=1, suffix_pages_width=0, prefix_len=1 << 19), 608 * 64),
    (dict(tokens=1216, q_heads=1, batch=1216, suffix_pages_width=8, prefix_len=0), 1216)], ids=["shared", "own"])
def test_ranges_are_bounded(lib, kw, rows):
    """Where one range of keys fills the SMs, 2^19 keys are four ranges of 2^17."""
    kw.update(k_heads=1, head_dim=8, page_size=1 << 16)
    for dtype in (BF16, FP16):
        assert lib.nf4_prefix_attention_workspace_size(args(dtype=dtype, **kw)) == rows * 4 * (8 * 4 + 8)


def test_scales_that_binary32_does_not_hold(lib):
    """The kernels work with scale * log2(e) in binary32, where it must neither vanish nor overflow."""
    log2e = 1.4426950408889634
    least, most = 2.0 ** -126 / log2e, (2.0 - 2.0 ** -23) * 2.0 ** 127 / log2e
    for scale in (5e-324, 1e-60, 1e-46, least * 0.999, most * 1.001, 1e300):
        assert lib.nf4_prefix_attention(args(scale=scale), A, 1 << 30, None) == ERR_SIZE, scale
        assert lib.nf4_prefix_attention_workspace_size(args(scale=scale)) == 0, scale
    for scale in (least * 1.001, 0.1, most * 0.999):
        assert lib.nf4_prefix_attention_workspace_size(args(scale=scale)) > 0, scale

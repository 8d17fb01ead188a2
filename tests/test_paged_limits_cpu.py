"""Calls on the 16-bit cache that are too large are refused on the host, before anything is launched."""
import pytest

from moe_decode_megakernel_persistent_gb300 import _lib as L
from tests.test_kv4_cpu import cache, code, rows
from tests.test_paged_cpu import lib, mass  # noqa: F401


@pytest.mark.parametrize("kw,heads,dtype", [
    (dict(max_pages=16777215, n_kv_heads=1), 1, L.MK_BF16),                       # spans of 256 positions pass 31 bits: few columns
    (dict(max_pages=16777215, n_kv_heads=1, rows=40), 1, L.MK_BF16),              # and many
    (dict(n_seqs=500000, max_pages=10000, n_kv_heads=1), 1, L.MK_F32),            # a block for every 256 positions
    (dict(n_seqs=13000, rows=40, max_pages=200000, n_kv_heads=2), 4, L.MK_BF16),  # items of the masses of many columns
    (dict(rows=524287, n_kv_heads=1024, max_pages=4, n_pages=64), 4096, L.MK_F32)])  # rows of q's parts
def test_masses_of_too_large_calls_are_refused(lib, kw, heads, dtype):  # noqa: F811
    c = cache(**kw)
    assert L.mk_paged_attention_bytes(c, heads, dtype, False) > 0 or kw == dict(max_pages=16777215, n_kv_heads=1)
    assert L.mk_paged_attention_bytes(c, heads, dtype, True) == 0
    m = mass(seq_stride=1 << 50, head_stride=1 << 32)
    got = code(L.mk_paged_attention, c, heads, rows(), dtype, 1.0, rows(), None, m, 0x8000, 1 << 62)
    assert got == L.MK_ERR_INVALID_ARG and "too large" in L.mk_last_error()


def test_masses_of_the_largest_calls_have_a_workspace(lib):  # noqa: F811
    for kw, heads, dtype in ((dict(max_pages=16777214, n_kv_heads=1), 1, L.MK_BF16),
                             (dict(rows=524256, n_kv_heads=1024, max_pages=4, n_pages=64), 4096, L.MK_BF16)):
        assert L.mk_paged_attention_bytes(cache(**kw), heads, dtype, True) > 0

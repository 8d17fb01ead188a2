"""The 16-bit cache's entry points: refusals on the host before any launch, sizes, and the
operators restated for the GPU tests."""
import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import _build
from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300 import paged
from tests import _paged as R
from tests.test_kv4_cpu import BAD, cache, code, rows


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return L.load()


def mass(**kw):
    return L.mk_paged_mass(**{**dict(data=0x9000, seq_stride=1 << 20, head_stride=1 << 10, decay=1.0), **kw})


def attention(c, heads=2, q=None, dtype=L.MK_BF16, scale=1.0, out=None, m=None, ws=0x8000, n=1 << 40):
    return code(L.mk_paged_attention, c, heads, q or rows(), dtype, scale, out or rows(), None, m, ws, n)


def evict(c, m=None, keep=16, recent=4, kept=0xA000, lengths=0xB000, to=None, ws=0x8000, n=1 << 40):
    return code(L.mk_paged_evict, c, m or mass(), keep, recent, kept, lengths, to or mass(data=0x90000000), ws, n)


@pytest.mark.parametrize("kw,want", BAD + [(dict(n_pages=1 << 22), L.MK_ERR_INVALID_ARG)])
def test_descriptions_are_refused_by_every_call(lib, kw, want):
    c = cache(**kw)
    assert code(L.mk_paged_store, c, rows(), rows(), L.MK_BF16) == want
    heads = 2000 if kw.get("n_kv_heads") == 2000 else 2
    assert attention(c, heads) == want
    assert L.mk_paged_attention_bytes(c, heads, L.MK_BF16) == L.mk_paged_attention_bytes(c, heads, L.MK_F32, True) == 0
    if kw == dict(max_pages=1 << 25):
        assert evict(c) == want and L.mk_paged_evict_bytes(c, 16) == 0
        assert evict(cache(max_pages=6145)) == L.MK_ERR_UNSUPPORTED and L.mk_paged_evict_bytes(cache(max_pages=6144), 16) > 0
    elif "rows" not in kw:                    # eviction has no rows
        if kw != dict(n_seqs=1000):
            assert evict(c) == want
            assert L.mk_paged_evict_bytes(c, 16) == 0
    assert L.mk_last_error()


def test_rows_types_and_masses_are_refused(lib):
    c, inv = cache(), L.MK_ERR_INVALID_ARG
    for bad in (rows(data=None), rows(data=0x4008), rows(head_stride=4), rows(row_stride=7), rows(seq_stride=1)):
        assert code(L.mk_paged_store, c, bad, rows(), L.MK_BF16) == inv
        assert code(L.mk_paged_store, c, rows(), bad, L.MK_BF16) == inv
        assert attention(c, q=bad) == inv and attention(c, out=bad) == inv
    for dt in (2, 3, -1):
        assert code(L.mk_paged_store, c, rows(), rows(), dt) == inv
        assert attention(c, dtype=dt) == inv
    for heads in (0, 3, -2, 8192):
        assert attention(c, heads) == inv
    for scale in (float("inf"), float("nan"), -float("inf"), 1e18, -2e30):
        assert attention(c, scale=scale) == inv
    two = cache(n_seqs=2)
    for m, why in ((mass(data=None), "NULL"), (mass(data=0x9004), "aligned"), (mass(seq_stride=-4), "stride"),
                   (mass(head_stride=258), "stride"), (mass(head_stride=252), "overlap"), (mass(seq_stride=1024), "overlap"),
                   (mass(decay=float("nan")), "finite"), (mass(decay=float("inf")), "finite")):
        assert attention(two, m=m) == inv and why in L.mk_last_error(), why
        if why != "finite":
            assert evict(two, m=m) == inv and why in L.mk_last_error()
            assert evict(two, to=m) == inv and why in L.mk_last_error()
    need = L.mk_paged_attention_bytes(c, 2, L.MK_BF16, True)
    assert need > 0
    for ws, n in ((0, need), (0x8008, need), (0x8000, need - 1)):
        assert attention(c, m=mass(), ws=ws, n=n) == inv and "workspace" in L.mk_last_error()


def test_evictions_are_refused(lib):
    c, inv = cache(), L.MK_ERR_INVALID_ARG
    for kw in (dict(keep=0), dict(keep=-1), dict(recent=-1), dict(recent=17), dict(kept=None), dict(lengths=None),
               dict(keep=1 << 30, recent=0), dict(ws=0), dict(ws=0x8008), dict(n=2 * 16 * 4 - 1)):
        assert evict(c, **kw) == inv, kw
    assert L.mk_paged_evict_bytes(c, 0) == 0 and L.mk_paged_evict_bytes(c, 16) > 0
    # the same memory with other strides is neither in place nor apart
    assert evict(c, to=mass(head_stride=2048)) == inv and "strides" in L.mk_last_error()


def test_calls_without_rows_launch_nothing(lib):
    for kw in (dict(n_seqs=0), dict(rows=0)):
        c = cache(pool=None, table=None, lengths=None, n_pages=0, **kw)
        assert code(L.mk_paged_store, c, None, None, L.MK_BF16) == L.MK_OK
        assert code(L.mk_paged_attention, c, 2, None, L.MK_F32, 1.0, None, None, None, 0, 0) == L.MK_OK
    c = cache(pool=None, table=None, lengths=None, n_pages=0, n_seqs=0)
    assert code(L.mk_paged_evict, c, None, 16, 0, None, None, None, 0, 0) == L.MK_OK


def test_pools_and_masses_of_zeros():
    for bad in ((0, 4, 128), (3, 0, 128), (3, 4, 96)):
        with pytest.raises(ValueError):
            paged.new_pool(*bad, device="cpu")
    assert paged.new_pool(3, 4, 64, device="cpu").shape == (3, 2, 4, 128, 64)
    assert paged.new_pool(3, 4, 128, n_layers=2, device="cpu").shape == (2, 3, 2, 4, 128, 128)
    m = paged.new_mass(torch.zeros((5, 3), dtype=torch.int32), 4)
    assert m.shape == (5, 4, 384) and m.dtype == torch.float32 and not m.any()


def test_the_restated_eviction():
    """By hand."""
    m = torch.tensor([3.0, 0.0, 1.0, 1.0, 2.0, 2.0, 0.5, 0.0])
    assert R.evict(m, 8, 4, 1) == [0, 4, 5, 7]         # slots 1, 2 and 3 take the late ones in order
    assert R.evict(m, 8, 5, 1) == [0, 5, 2, 7, 4]      # 0, 4, 5, then the tie of 2 and 3 goes to 2; 7 is recent
    assert R.evict(m, 3, 5, 1) == [0, 1, 2, -1, -1]
    assert R.evict(m, 8, 3, 3) == [5, 6, 7]
    assert R.evict(torch.tensor([1.0, float("nan"), 5.0, float("nan")]), 4, 2, 0) == [3, 1]

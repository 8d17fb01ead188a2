"""The 4-bit cache's and the page copy's entry points: refusals on the host
before any launch, sizes, and the format restated for the GPU tests."""
import ctypes as C

import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import _build
from moe_decode_megakernel_persistent_gb300 import _lib as L
from tests import _kv4 as R


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return L.load()


def cache(**kw):
    f = dict(pool=0x1000, table=0x2000, lengths=0x3000, n_new=None, status=None, n_pages=4, n_kv_heads=2, head_dim=64,
             n_seqs=1, max_pages=2, rows=1)
    f.update(kw)
    return L.mk_kv4_cache(**f)


def rows(**kw):
    return L.mk_kv4_rows(**{**dict(data=0x4000, seq_stride=0, row_stride=0, head_stride=64), **kw})


def code(f, *a):
    try:
        f(*a)
        return L.MK_OK
    except L.MKError as e:
        return e.code


BAD = [(dict(head_dim=96), L.MK_ERR_UNSUPPORTED), (dict(head_dim=256), L.MK_ERR_UNSUPPORTED)] + [
    (k, L.MK_ERR_INVALID_ARG) for k in (
        dict(n_kv_heads=0), dict(n_kv_heads=2000), dict(n_seqs=-1), dict(rows=-1), dict(n_pages=0), dict(max_pages=0),
        dict(max_pages=1 << 25), dict(n_seqs=1000, rows=1000), dict(pool=None), dict(pool=0x1008), dict(table=None),
        dict(lengths=None))]


@pytest.mark.parametrize("kw,want", BAD)
def test_descriptions_are_refused_by_every_call(lib, kw, want):
    c = cache(**kw)
    assert code(L.mk_kv4_store, c, rows(), rows(), L.MK_BF16) == want
    assert code(L.mk_kv4_load, c, rows(), rows(), L.MK_BF16) == want
    assert code(L.mk_kv4_attention, c, 2 if kw.get("n_kv_heads") != 2000 else 2000, rows(), L.MK_BF16, 1.0, rows(), None,
                0x8000, 1 << 40) == want
    assert L.mk_kv4_attention_bytes(c, 2, L.MK_BF16) == 0
    assert L.mk_last_error()


def test_rows_and_types_are_refused(lib):
    c, inv = cache(), L.MK_ERR_INVALID_ARG
    for bad in (rows(data=None), rows(data=0x4008), rows(head_stride=4), rows(row_stride=7), rows(seq_stride=1)):
        assert code(L.mk_kv4_store, c, bad, rows(), L.MK_BF16) == inv
        assert code(L.mk_kv4_store, c, rows(), bad, L.MK_BF16) == inv
        assert code(L.mk_kv4_load, c, bad, rows(), L.MK_BF16) == inv
        assert code(L.mk_kv4_attention, c, 2, bad, L.MK_BF16, 1.0, rows(), None, 0x8000, 1 << 40) == inv
        assert code(L.mk_kv4_attention, c, 2, rows(), L.MK_BF16, 1.0, bad, None, 0x8000, 1 << 40) == inv
    for dt in (2, 3, -1):
        assert code(L.mk_kv4_store, c, rows(), rows(), dt) == inv
        assert code(L.mk_kv4_attention, c, 2, rows(), dt, 1.0, rows(), None, 0x8000, 1 << 40) == inv
    for heads in (0, 3, -2, 8192):
        assert code(L.mk_kv4_attention, c, heads, rows(), L.MK_BF16, 1.0, rows(), None, 0x8000, 1 << 40) == inv
    for scale in (float("inf"), float("nan"), -float("inf"), 1e18, -2e30):
        assert code(L.mk_kv4_attention, c, 2, rows(), L.MK_BF16, scale, rows(), None, 0x8000, 1 << 40) == inv
    assert code(L.mk_kv4_store, None, rows(), rows(), L.MK_BF16) == inv
    # a workspace that is missing, misaligned or too small
    assert L.mk_kv4_attention_bytes(c, 2, L.MK_BF16) == 0      # short work needs none
    c = cache(n_pages=1 << 20, max_pages=1 << 20)
    need = L.mk_kv4_attention_bytes(c, 2, L.MK_BF16)
    assert need > 0
    for ws, n in ((0, need), (0x8008, need), (0x8000, need - 1)):
        assert code(L.mk_kv4_attention, c, 2, rows(), L.MK_BF16, 1.0, rows(), None, ws, n) == inv
        assert "workspace" in L.mk_last_error()


def test_calls_without_rows_launch_nothing(lib):
    """Nothing is read, so no address is needed (and this machine has no GPU to launch on)."""
    for kw in (dict(n_seqs=0), dict(rows=0)):
        c = cache(pool=None, table=None, lengths=None, n_pages=0, **kw)
        assert code(L.mk_kv4_store, c, None, None, L.MK_BF16) == L.MK_OK
        assert code(L.mk_kv4_load, c, None, None, L.MK_F32) == L.MK_OK
        assert code(L.mk_kv4_attention, c, 2, None, L.MK_F32, 1.0, None, None, 0, 0) == L.MK_OK


def test_page_sizes(lib):
    assert L.mk_kv4_page_bytes(4, 128) == 4 * R.record(128) == 4 * 17408
    assert L.mk_kv4_page_bytes(2, 64) == 2 * R.record(64) == 2 * 8704
    assert L.mk_kv4_page_bytes(0, 64) == L.mk_kv4_page_bytes(1, 80) == 0


def test_page_copy_refuses_moves_that_meet(lib):
    f = lambda src, dst, **kw: code(L.mk_page_copy, *{**dict(pool=0x1000, layers=2, pages=8, size=32), **kw}.values(), src, dst)
    for src, dst in (([0], [8]), ([8], [0]), ([-1], [0]), ([0], [-1]), ([0, 1], [2, 2]), ([0, 1], [1, 2]), ([2], [2]),
                     ([5, 6, 7], [0, 1, 5])):
        assert f(src, dst) == L.MK_ERR_INVALID_ARG, (src, dst)
    for kw in (dict(pool=None), dict(pool=0x1004), dict(layers=0), dict(pages=0), dict(size=24), dict(size=0), dict(size=1 << 41)):
        assert f([0], [1], **kw) == L.MK_ERR_INVALID_ARG, kw
    assert f([], []) == L.MK_OK
    with pytest.raises(ValueError):
        f([0, 1], [2])


def test_the_restated_format(lib):
    """By hand: a group of 64 whose largest value is 3.5 has scale 0.5; halves go to even; the sign is bit 3."""
    x = torch.zeros(64)
    x[:6] = torch.tensor([3.5, -3.5, 0.25, 0.75, -0.25, -1.2])
    c, s = R.quantise(x)
    assert s.tolist() == [0.5] and c[:6].tolist() == [7, 15, 0, 2, 0, 10] and not c[6:].any()
    assert R.values(c, s)[:6].tolist() == [3.5, -3.5, 0, 1, 0, -1]
    pool = torch.zeros((2, 1, R.record(64)), dtype=torch.uint8)
    R.put(pool, 64, 1, 70, 0, 1, c, s)
    at = 4352 + 2176 + 6 * 32                 # second tile, V half, row 6
    assert pool[1, 0, at:at + 3].tolist() == [7 + 15 * 16, 2 * 16, 10 * 16]
    assert pool[1, 0, 4352 + 2176 + 2048 + 12: 4352 + 2176 + 2048 + 14].tolist() == [0x00, 0x3F]
    got = R.get(pool, 64, 1, 70, 0, 1)
    assert torch.equal(got[0], c) and torch.equal(got[1], s)
    k = torch.randn(200, 1, 64)
    R.fill(pool, 64, torch.tensor([1, 0]), k, -k)
    kk, vv = R.cache_values(pool, 64, torch.tensor([1, 0]), 200)
    assert torch.equal(kk, R.values(*R.quantise(k))) and torch.equal(vv, -kk)
    for p in (0, 63, 64, 127, 128, 199):
        assert torch.equal(R.values(*R.get(pool, 64, [1, 0][p // 128], p % 128, 0, 0)), kk[p, 0])

"""Host side of the page calls: null contexts, and prefix reuse to the token
over a fake engine."""
import ctypes as C

import pytest

from moe_decode_megakernel_persistent_gb300 import _build
from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300.engine import PrefixCache
from tests.test_prefix_cache_cpu import FakeEngine, _prompt


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return L.load()


def test_null_contexts_are_refused(lib):
    moved = C.c_int32(7)
    assert lib.mk_kv_alloc_fmt(None, 4, L.MK_BF16) == L.MK_ERR_INVALID_ARG
    assert lib.mk_seq_fork_at(None, 0, 1, 5, None) == L.MK_ERR_INVALID_ARG
    assert lib.mk_seq_truncate(None, 0, 5, None) == L.MK_ERR_INVALID_ARG
    assert lib.mk_kv_compact(None, C.byref(moved), None) == L.MK_ERR_INVALID_ARG and moved.value == 0
    assert lib.mk_kv_compact(None, None, None) == L.MK_ERR_INVALID_ARG


class ForkAtEngine(FakeEngine):
    def fork_at(self, src, dst, n_tokens):
        self.calls.append(("fork_at", src, dst, n_tokens))


def test_prefixes_are_reused_to_the_token():
    e = ForkAtEngine()
    pc = PrefixCache(e, capacity=4, whole_pages=False)
    a = _prompt(1, 8022)
    pc.prefill(0, a)
    pc.keep(0, a.tolist())
    e.calls.clear()
    _, n = pc.prefill(1, a)                       # one token is left to prefill: it gives the next one
    assert n == 8021 and e.calls == [("fork_at", 0, 1, 8021), ("prefill", 1, 8021, 1)]
    e.calls.clear()
    _, n = pc.prefill(2, a[:7])
    assert n == 6 and e.calls == [("fork_at", 0, 2, 6), ("prefill", 2, 6, 1)]
    e.calls.clear()
    b = a.clone()
    b[0] += 1
    _, n = pc.prefill(3, b)
    assert n == 0 and e.calls == [("prefill", 3, 0, 8022)]

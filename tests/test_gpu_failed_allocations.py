"""A refused allocation leaves nothing behind: what is called next works, or is refused in its turn."""
import pytest
import torch

import synth
from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300.engine import Engine
from synth import weights as SW
from tests import _kv4 as R

pytestmark = pytest.mark.gpu

TINY = synth.CONFIGS[1].model


@pytest.fixture(scope="module")
def tiny():
    m = TINY.with_(wdtype="int4")
    return m, SW.model_torch(m, "cuda")


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_a_pool_that_is_too_large_then_a_small_one(gpu_lib, tiny, fmt, monkeypatch):
    """The out-of-memory error of the first is not taken for one of the launches that follow."""
    m, w = tiny
    alloc, tried = L.mk_kv_alloc_fmt, []

    def twice(ctx, n_pages, f):
        with pytest.raises(L.MKError) as e:
            alloc(ctx, 1 << 30, f)                   # some 100 TB
        assert e.value.code == L.MK_ERR_CUDA
        tried.append(1)
        alloc(ctx, n_pages, f)

    monkeypatch.setattr(L, "mk_kv_alloc_fmt", twice)
    eng = Engine(m, w, n_pages=8, max_ctx=1024, max_seqs=2, kv_dtype=fmt)
    assert tried
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = torch.randn((m.n_layers, 200, 2, m.n_kv_heads, m.head_dim), generator=g, device="cuda").to(torch.bfloat16)
    eng.kv_write(0, 0, kv)
    assert eng.info()["free_pages"] == 6
    want = kv if fmt == "bf16" else R.values(*R.quantise(kv)).to(torch.bfloat16)
    assert torch.equal(eng.kv_read(0, 0, 200), want)
    eng.sync()
    eng.close()

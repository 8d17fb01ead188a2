"""The workspace of prompt chunks is made by the first chunk that needs it.  Where the GPU has no
room for it, that chunk is refused, and so is the next: neither launches on a half-made one.  With
room again a chunk gives what it gives in a context that never failed."""
import pytest
import torch

import synth
from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300.engine import Engine
from synth import prompts as SP
from synth import weights as SW

pytestmark = pytest.mark.gpu

TINY = synth.CONFIGS[1].model


def take_all_but(left):
    """Tensors that hold the GPU's free memory but for about `left` bytes."""
    held, size = [], 1 << 34
    torch.cuda.empty_cache()
    while size >= 1 << 21:
        if torch.cuda.mem_get_info()[0] - size < left:
            size >>= 1
            continue
        try:
            held.append(torch.empty(size, dtype=torch.uint8, device="cuda"))
        except torch.cuda.OutOfMemoryError:
            size >>= 1
    return held


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
@pytest.mark.parametrize("left", [32 << 20, 96 << 20])
def test_a_chunk_without_room_is_refused_until_there_is_some(gpu_lib, fmt, left):
    m = TINY.with_(wdtype="int4")
    w = SW.model_torch(m, "cuda")
    p = torch.from_numpy(SP.prompt_tokens(m.seed, m.vocab, 300, seq=1)).cuda()

    def engine():
        return Engine(m, w, n_pages=8, max_ctx=1024, max_seqs=2, kv_dtype=fmt)

    eng = engine()
    want = eng.prefill(0, p).item()
    kv = eng.kv_read(0, 0, 300).clone()
    eng.sync()
    eng.close()

    eng = engine()
    out = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = take_all_but(left)
    try:
        for _ in range(2):
            with pytest.raises(L.MKError) as e:
                eng.prefill(0, p, out=out)
            assert e.value.code == L.MK_ERR_CUDA and eng.seq_length(0) == -1 and eng.info()["free_pages"] == 8
    finally:
        del held
        torch.cuda.empty_cache()
    assert eng.prefill(0, p, out=out).item() == want
    assert torch.equal(eng.kv_read(0, 0, 300).view(torch.int16), kv.view(torch.int16))
    eng.sync()
    eng.close()

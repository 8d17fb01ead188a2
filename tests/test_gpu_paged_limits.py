"""The operators on the 16-bit paged cache at the ends of what their arguments may be."""
import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import paged
from tests.test_gpu_paged import i32, make, masses

pytestmark = pytest.mark.gpu


def test_an_eviction_that_keeps_2_31_positions(gpu_lib):
    """The largest keep: the positions of a table of 300, and a list of 8.6 GB whose rest is -1."""
    keep = 2 ** 31 - 1
    pool, table = make([300], 1, 64, seed=50)
    before, m = pool.clone(), masses(table, 1)
    kept, lengths, new = paged.evict(pool, table, i32([300]), m, keep, recent=7)
    assert kept.shape == (1, 1, keep) and lengths.tolist() == [300]
    assert torch.equal(kept[0, 0, :300], torch.arange(300, dtype=torch.int32, device="cuda"))
    for part in kept[0, 0, 300:].split(1 << 28):
        assert int(part.min()) == int(part.max()) == -1
    assert torch.equal(new[..., :300], m[..., :300]) and not new[..., 300:].any()
    assert torch.equal(pool.view(torch.int16), before.view(torch.int16))
    del kept, part
    torch.cuda.empty_cache()

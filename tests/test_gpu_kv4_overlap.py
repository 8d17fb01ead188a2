"""Attention's out may not lie in the pool that the call reads."""
import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import kv4
from tests.test_gpu_kv4 import BF, F32, i32, make, rows_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 40])
def test_out_may_not_be_the_pools_memory(gpu_lib, dtype, rows):
    pool, table = make([100], 2, 64, seed=28)
    q = rows_of(1, rows, 4, 64, dtype)
    want = kv4.attention(q, pool, table, i32([100]))
    # the pool and the tensor behind it in one allocation
    whole = torch.zeros(pool.numel() + q.numel() * q.element_size(), dtype=torch.uint8, device="cuda")
    inside = whole[:pool.numel()].view(pool.shape)
    inside.copy_(pool)
    for at in (0, 16, pool.numel() - 16):
        out = whole[at:at + q.numel() * q.element_size()].view(dtype).view(q.shape)
        with pytest.raises(ValueError, match="out must not overlap the pool"):
            kv4.attention(q, inside, table, i32([100]), out=out)
    assert torch.equal(inside, pool)
    out = whole[pool.numel():].view(dtype).view(q.shape)
    assert kv4.attention(q, inside, table, i32([100]), out=out) is out and torch.equal(out, want)

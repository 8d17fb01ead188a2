"""Page moves on the GPU against torch's indexing."""
import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300 import pages

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,dtype,n", [((3, 9, 2, 4, 128, 128), torch.bfloat16, 4), ((1, 3, 16), torch.uint8, 1),
                                           ((49, 40, 4, 8704), torch.uint8, 19), ((2, 1201, 24), torch.float32, 600),
                                           ((5, 4, 16384 + 16), torch.uint8, 2), ((1, 2, 3, 40000), torch.int64, 1)])
def test_pages_move_in_every_layer(gpu_lib, shape, dtype, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    size = torch.empty((), dtype=dtype).element_size()
    pool = torch.randint(0, 256, (*shape[:-1], shape[-1] * size), dtype=torch.uint8, device="cuda", generator=g).view(dtype)
    order = torch.randperm(shape[1], generator=torch.Generator().manual_seed(n)).tolist()
    src, dst = order[:n], order[n:2 * n]
    want = pool.view(torch.uint8).clone()
    want[:, dst] = want[:, src]
    pages.copy(pool, src, dst)
    assert torch.equal(pool.view(torch.uint8), want)
    # one source for several destinations
    if shape[1] > 2:
        pages.copy(pool, [order[0]] * 2, [order[-1], order[-2]])
        want[:, order[-1]] = want[:, order[-2]] = want[:, order[0]]
        assert torch.equal(pool.view(torch.uint8), want)
    pages.copy(pool, [], [])
    assert torch.equal(pool.view(torch.uint8), want)


def test_offsets_past_32_bits(gpu_lib):
    pool = torch.zeros((3, 5, 1 << 29), dtype=torch.uint8, device="cuda")      # 7.5 GB
    pool[:, 4, -1] = 9
    pool[2, 1] = 3
    pages.copy(pool, [4, 1], [0, 3])
    assert pool[:, 0, -1].tolist() == [9, 9, 9] and int(pool[:, 0].max()) == 9
    assert (pool[2, 3] == 3).all() and not pool[0, 3].any()


def test_refusals(gpu_lib):
    pool = torch.zeros((2, 4, 32), dtype=torch.uint8, device="cuda")
    for src, dst in (([0], [4]), ([-1], [0]), ([0, 1], [2, 2]), ([0, 1], [1, 2]), ([3], [3])):
        with pytest.raises(L.MKError) as e:
            pages.copy(pool, src, dst)
        assert e.value.code == L.MK_ERR_INVALID_ARG
    for p, src, dst in ((pool.cpu(), [0], [1]), (pool[0], [0], [1]), (pool[:, :, ::2], [0], [1]), (pool, [0], [1, 2])):
        with pytest.raises(ValueError):
            pages.copy(p, src, dst)
    with pytest.raises(L.MKError):
        pages.copy(torch.zeros((2, 4, 24), dtype=torch.uint8, device="cuda"), [0], [1])   # 24-byte pages
    assert not pool.any()

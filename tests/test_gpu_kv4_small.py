"""Stores and loads whose rows are fewer parts than a warp has threads, and
head counts whose parts do not fill a block evenly: codes byte by byte against
tests/_kv4.py, nothing else written."""
import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import kv4
from tests import _kv4 as R
from tests.test_gpu_kv4 import BF, F32, gen, i32, table_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hd,G", [(64, 1), (128, 1), (64, 5), (64, 33), (128, 17)])
@pytest.mark.parametrize("lengths,rows", [([1], 1), ([129, 3], 2), ([40, 700, 0], 33)])
def test_rows_of_any_number_of_heads(gpu_lib, hd, G, dtype, lengths, rows):
    table, n_pages = table_for(lengths, seed=G)
    pool = torch.randint(0, 256, (n_pages, G, R.record(hd)), dtype=torch.uint8, device="cuda", generator=gen(G))
    k, v = (torch.randn((len(lengths), rows, G, hd), device="cuda", generator=gen(j)).to(dtype) for j in (3, 4))
    want = pool.cpu().clone()
    for i, ln in enumerate(lengths):
        for r in range(max(0, rows - ln), rows):
            p = ln - rows + r
            for kv, x in enumerate((k, v)):
                code, s = R.quantise(x[i, r].cpu())
                for g in range(G):
                    R.put(want, hd, int(table[i, p // R.PAGE]), p % R.PAGE, g, kv, code[g], s[g])
    kv4.store(pool, table, i32(lengths), k, v)
    assert torch.equal(pool.cpu(), want)
    for got, x in zip(kv4.load(pool, table, i32(lengths), rows, dtype=F32), (k, v)):
        ref = R.values(*R.quantise(x))
        for i, ln in enumerate(lengths):
            ref[i, :max(0, rows - ln)] = 0
        assert torch.equal(got, ref.float())

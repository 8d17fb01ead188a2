"""Attention over the 4-bit cache next to values far larger than the rest: a row
that does not see such a position has the error of a cache without it, whatever
the other rows of the call see.  The reference and the bounds are those of
tests/_kv4.py, with the largest V taken over what the rows in question see."""
import math

import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import kv4
from tests import _kv4 as R
from tests.test_gpu_kv4 import BF, F32, i32, poisoned_pool, rows_of, table_for

pytestmark = pytest.mark.gpu


def check_rows(q, kc, vc, out, lse, first, lo, hi, scale):
    """Rows lo .. hi - 1, whose positions are first + lo .. first + hi - 1."""
    n, hd = first + hi, q.shape[-1]
    o, l, A, D = R.attend(q[0, lo:hi], kc[:n], vc[:n], first + lo, scale)
    inner, half, le = R.bounds(A, D, l, n, hd, q.dtype, float(vc[:n].abs().max()))
    off = (out[0, lo:hi].double() - o).abs() - (inner * (1 + half) + half * o.abs())
    assert off.max() <= 0, (lo, hi, off.max().item())
    assert ((lse[0, lo:hi].double() - l).abs() <= le).all(), (lo, hi, ((lse[0, lo:hi].double() - l).abs() - le).max().item())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("dtype,rows,H,G", [
    (BF, 20, 4, 1), (BF, 33, 4, 4), (BF, 40, 4, 1), (F32, 40, 4, 1), (BF, 130, 2, 1), (F32, 130, 2, 1),   # tiles of 128 columns
    *((t, *c) for t in (BF, F32) for c in ((2, 1, 1), (5, 4, 1), (8, 8, 2))), (F32, 20, 4, 1), (F32, 33, 4, 4)])
@pytest.mark.parametrize("power", [8, 14, 20])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_rows_that_do_not_see_an_outlier(gpu_lib, dtype, hd, rows, H, G, power, which):
    """The last position but one is 2^power times the rest: only the last two rows see it."""
    n = 700
    table, n_pages = table_for([n])
    pool = poisoned_pool(n_pages, G, hd)
    g = torch.Generator(device="cuda").manual_seed(power)
    k, v = (torch.randn((n, G, hd), device="cuda", generator=g) for _ in range(2))
    for x, name in ((k, "k"), (v, "v")):
        if which in (name, "both"):
            x[n - 2] *= 2.0 ** power
    R.fill(pool, hd, table[0].long()[:-(-n // R.PAGE)], k, v)
    q = rows_of(1, rows, H, hd, dtype)
    out, lse = kv4.attention(q, pool, table, i32([n]), return_lse=True)
    kc, vc = R.cache_values(pool, hd, table[0].long(), n)
    scale = 1 / math.sqrt(hd)
    if rows > 2:
        check_rows(q, kc, vc, out, lse, n - rows, 0, rows - 2, scale)
    check_rows(q, kc, vc, out, lse, n - rows, rows - 2, rows, scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [4, 40])
def test_growing_values_stay_with_who_sees_them(gpu_lib, dtype, rows):
    """V doubles with every position that the call adds, so that each row sees a larger one than the row before."""
    n, hd, H = 300, 64, 4
    table, n_pages = table_for([n])
    pool = poisoned_pool(n_pages, 1, hd)
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v = (torch.randn((n, 1, hd), device="cuda", generator=g) for _ in range(2))
    v[n - 20:] *= 2.0 ** torch.arange(1, 21, device="cuda")[:, None, None]
    R.fill(pool, hd, table[0].long()[:-(-n // R.PAGE)], k, v)
    q = rows_of(1, rows, H, hd, dtype)
    out, lse = kv4.attention(q, pool, table, i32([n]), return_lse=True)
    kc, vc = R.cache_values(pool, hd, table[0].long(), n)
    for r in range(rows):
        check_rows(q, kc, vc, out, lse, n - rows, r, r + 1, 1 / math.sqrt(hd))

"""What the operators on the 16-bit paged cache make of values: the bits of bf16 rows' weights,
infinite keys, values and queries."""
import math

import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import paged
from tests import _paged as R
from tests.test_gpu_paged import BF, F32, check, i32, make, masses, randn

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- weights of bf16 rows

@pytest.mark.parametrize("hd,rows,seqs,width", [
    (128, 1, 1, None), (128, 4, 1, None), (128, 6, 1, None), (64, 8, 1, None), (64, 1, 1, None),   # clusters, 4 to 32 columns
    (128, 1, 700, None), (64, 7, 300, None),                                                      # equal runs
    (128, 40, 1, None), (64, 60, 3, None),                                                        # one tile of 128 columns a block
    (128, 60, 1, 2000), (64, 64, 2, 2000)])                                                       # two
def test_weights_of_bf16_rows_have_16_bits(gpu_lib, hd, rows, seqs, width):
    """Values of V are +-1, whose sums nearly cancel, so that an output's own rounding is small next to what a
    weight of 8 bits would be off by (2^-9 / sqrt(3 n) of the weights' sum, 1, as a norm: 1e-4 at n = 100).  A score is
    one product, exact, then scaled and taken from the maximum with an error of a few 2^-24 of magnitudes up to 2:
    with the exponential's 2^-22 a weight is off by 2^-20, which enters twice.  Each of the 2 n terms of the sums
    of two parts is cut off by 2^-23 of the sum at most, each of the n terms below by 2^-24; two parts of a weight leave 2^-16."""
    n = max(100, rows + 20)
    G, H = 2, 8
    pool, table = make([n] * seqs, G, hd, seed=30, width=width)
    ones = torch.where(randn((2, n, G, hd), 31) < 0, -1.0, 1.0)
    k = torch.zeros((n, G, hd), device="cuda")
    k[..., 0] = randn((n, G), 32).clamp(-2, 2)
    for i in range(seqs):
        R.put(pool, table, i, 0, k, ones[i % 2])
    q = torch.zeros((seqs, rows, H, hd), dtype=BF, device="cuda")
    q[..., 0] = (1 + torch.rand((seqs, rows, H), device="cuda", generator=torch.Generator(device="cuda").manual_seed(33)))
    out = paged.attention(q, pool, table, i32([n] * seqs), scale=0.5)
    inner = 2 * 2.0 ** -20 + 2 * n * 2.0 ** -23 + n * 2.0 ** -24 + 2.0 ** -16
    for i in sorted({0, 1, seqs // 2, seqs - 1} & set(range(seqs))):
        want, _, _, A, _ = R.attend(q[i], *R.rows_of(pool, table, i, n), n - rows, 0.5)
        assert bool(((A - 1).abs() < 1e-12).all())
        err = (out[i].double() - want).abs()
        assert bool((err <= inner + (want.abs() + inner) * 2.0 ** -8).all()), (i, float((err / (inner + want.abs() * 2.0 ** -8)).max()))


# ---------------------------------------------------------------- infinities

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,n_new", [(1, None), (9, None), (40, None), (150, None), (150, [131]), (257, [256])])
def test_masses_of_keys_of_minus_infinity(gpu_lib, dtype, hd, rows, n_new):
    """Positions whose scores are all -infinity receive nothing, next to columns that are none (a tile's padding,
    rows behind n_new), whose queries are taken as 0: 0 times infinity is NaN."""
    n = 600
    pool, table = make([n], 1, hd, seed=34)
    k = torch.zeros((n, 1, hd), device="cuda")
    k[:, :, 0] = randn((n, 1), 4)
    gone = torch.zeros(n, dtype=torch.bool, device="cuda")
    gone[5:90] = gone[250:260] = gone[300:310] = True
    k[gone, :, 0] = -math.inf
    R.put(pool, table, 0, 0, k, randn((n, 1, hd), 5))
    q = torch.zeros((1, rows, 2, hd), dtype=dtype, device="cuda")
    q[..., 0] = 1 + randn((1, rows, 2), 6).abs()
    m = masses(table, 1)
    _, _, got = check(q, pool, table, [n], n_new=n_new, scale=1.0, left_out=[gone], mass=m, decay=0.5)
    old = gone & (torch.arange(n, device="cuda") < n - (rows if n_new is None else n_new[0]))
    assert torch.equal(got[0, 0, :n][old], 0.5 * m[0, 0, :n][old])
    k[:, :, 0] = -math.inf                     # no score has a weight: old masses fade, new positions have none
    R.put(pool, table, 0, 0, k, randn((n, 1, hd), 5))
    got = m.clone()
    out, lse = paged.attention(q, pool, table, i32([n]), n_new=None if n_new is None else i32(n_new), scale=1.0, return_lse=True, mass=got, decay=0.5)
    assert not out.any() and bool((lse == -math.inf).all())
    first = n - (rows if n_new is None else n_new[0])
    assert torch.equal(got[0, 0, :first], 0.5 * m[0, 0, :first]) and not got[0, 0, first:n].any()
    assert torch.equal(got[0, 0, n:], m[0, 0, n:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("heavy_first", [False, True])
@pytest.mark.parametrize("light", [0.0, -math.inf])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,lengths", [(1, [2049]), (3, [700]), (1, [60000]), (1, [6000] * 40), (3, [30000, 900]), (40, [9000]), (100, [3000, 20000])])
def test_infinite_values_of_hardly_any_weight(gpu_lib, dtype, light, heavy_first, hd, rows, lengths):
    """An infinite V reaches its dimension however the work is cut, where its position's weight (2^-432 of the largest,
    or none) and that of every position of its block are below all fp32."""
    G, H = 2, 4
    pool, table = make(lengths, G, hd, seed=35)
    at = torch.arange(max(lengths), device="cuda")
    bad = {3: math.inf, 4: -math.inf, 9: math.nan}
    v = randn((max(lengths), G, hd), 36)
    for i, n in enumerate(lengths):
        k = torch.zeros((n, G, hd), device="cuda")
        first = n - max(rows, 8)               # (what all rows see)
        heavy = at[:n] < first // 2 if heavy_first else at[:n] >= first // 2
        k[..., 0] = torch.where(heavy, 300.0, light)[:, None]
        vi = v[:n].clone()
        for j, (d, x) in enumerate(bad.items()):
            vi[(first - 5 if heavy_first else 5) + j, :, d] = x
        R.put(pool, table, i, 0, k, vi)
    q = torch.zeros((len(lengths), rows, H, hd), dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    out = paged.attention(q, pool, table, i32(lengths), scale=1.0)
    for d, x in bad.items():
        assert bool((out[..., d].isnan() if math.isnan(x) else out[..., d] == x).all()), (d, out[..., d].flatten()[:8])
    rest = [d for d in range(hd) if d not in bad]
    assert bool(torch.isfinite(out[..., rest]).all())
    for i, n in list(enumerate(lengths))[:2]:
        k, vv = R.rows_of(pool, table, i, n)
        gone = k[:, 0, 0] == -math.inf
        want, wl, w, A, D = R.attend(q[i], k, torch.where(torch.isfinite(vv), vv, 0.0), n - rows, 1.0, gone)
        inner, half, _ = R.bounds(A, D, wl, n, hd, dtype)
        err = (out[i].double() - want).abs()[..., rest]
        assert bool((err <= (inner + (want.abs() + inner) * half)[..., rest]).all())


@pytest.mark.parametrize("rows", [1, 5, 150])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_query(gpu_lib, rows, sign):
    """An fp32 q that is infinite, against keys whose sign makes every score -infinity (no weight) or, for one
    position, +infinity (the rows that see it are NaN), as the products of whole fp32 numbers have it."""
    n, hd = 400, 64
    pool, table = make([n], 1, hd, seed=37)
    k = torch.zeros((n, 1, hd), device="cuda")
    k[:, :, 0] = -sign * (1 + randn((n, 1), 38).abs())
    k[:, :, 1:] = 1 + randn((n, 1, hd - 1), 39).abs()
    R.put(pool, table, 0, 0, k, randn((n, 1, hd), 40))
    q = randn((1, rows, 2, hd), 41)
    q[..., 0] = sign * math.inf
    m = masses(table, 1)
    m0 = m.clone()
    out, lse = paged.attention(q, pool, table, i32([n]), scale=1.0, return_lse=True, mass=m)
    assert not out.any() and bool((lse == -math.inf).all())
    assert torch.equal(m[..., :n - rows], m0[..., :n - rows]) and not m[..., n - rows:n].any()
    out, lse = paged.attention(q, pool, table, i32([n]), scale=-1.0, return_lse=True)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())


@pytest.mark.parametrize("rows,seqs", [(1, 19), (6, 19), (40, 19), (64, 38)])
def test_long_sums_of_one_sign_of_bf16_rows(gpu_lib, rows, seqs):
    """Runs of whole items of 131072 positions (pages in common) and V above 0: what the products cut off adds up.  An
    output's own rounding is off by 2^-8 at most, evenly to both sides: as a mean over 1024 dimensions of sizes over
    an octave 2^-8 / sqrt(3 x 1024), of which six times that are allowed.  Many columns: 4096 positions' 512 products cut
    off up to 2^-23 of their sum each, 32 such sums are added with 2^-24 (all in one sum: 9.2e-4 off).  Few: each of four
    warps adds the 4096 products of its positions, of which a product cuts off 2^-23 of the sum so far, a half of the whole."""
    n, hd, G = 131072, 128, 8
    pool = randn((512, 2, G, 128, hd), 60, BF)
    size = torch.exp2(torch.rand((G, 1, hd), device="cuda", generator=torch.Generator(device="cuda").manual_seed(61)))
    pool[:, 1] = (pool[:, 1].float().abs() * size).to(BF)
    table = torch.randint(0, 512, (seqs, n // 128), dtype=torch.int32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(62))
    q = randn((seqs, rows, 4 * G, hd), 63, BF, 1.5)
    out = paged.attention(q, pool, table, i32([n] * seqs))
    k, v = R.rows_of(pool, table, seqs - 1, n)
    want = torch.cat([R.attend(q[-1, :, 4 * g:4 * g + 4], k[:, g:g + 1], v[:, g:g + 1], n - rows, 1 / math.sqrt(hd))[0] for g in range(G)], 1)
    most = (512 + 16 if rows > 8 else 4096 / 2) * 2.0 ** -23 + 6 * 2.0 ** -8 / math.sqrt(3 * 1024)
    assert abs(float(((out[-1].double() - want) / want).mean())) < most


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,n", [(1, 30), (1, 40000), (5, 700), (40, 9000), (200, 2100)])
def test_large_values(gpu_lib, dtype, rows, n):
    """V of magnitudes 2^93 to 2^95: sums over the positions, by weights up to 2^8, stay in fp32."""
    pool, table = make([n], 2, 64, seed=42)
    v = torch.exp2(93 + 2 * torch.rand((n, 2, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(43)))
    k = randn((n, 2, 64), 44)
    R.put(pool, table, 0, 0, k, torch.where(k < 0, -v, v).clamp(-2.0 ** 95, 2.0 ** 95))
    check(randn((1, rows, 4, 64), 45, dtype), pool, table, [n], scale=0.5)


# ---------------------------------------------------------------- masses behind the ends, long sums

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,n_new", [(1, None), (5, [5, 0, 2, 5]), (60, [60, 1, 0, 33])])
def test_masses_behind_the_ends_are_not_used(gpu_lib, dtype, rows, n_new):
    """Behind a sequence's end and in its new positions masses are NaN: kept as they are there, not used here."""
    lengths = [300, 130, 1, 257]
    pool, table = make(lengths, 2, 64, seed=46, width=4)
    m = masses(table, 2)
    for i, n in enumerate(lengths):
        m[i, :, max(0, n - (rows if n_new is None else n_new[i])):] = math.nan
    q = randn((4, rows, 4, 64), 47, dtype)
    got = m.clone()
    paged.attention(q, pool, table, i32(lengths), n_new=None if n_new is None else i32(n_new), mass=got, decay=0.5)
    m[:] = torch.where(m.isnan(), 0.0, m)
    want = m.clone()
    paged.attention(q, pool, table, i32(lengths), n_new=None if n_new is None else i32(n_new), mass=want, decay=0.5)
    for i, n in enumerate(lengths):
        assert torch.equal(got[i, :, :n], want[i, :, :n]) and bool(torch.isfinite(got[i, :, :n]).all())
        assert bool(got[i, :, n:].isnan().all())


@pytest.mark.parametrize("rows", [40, 1])
def test_long_sums_of_one_sign(gpu_lib, rows):
    """152 items of 30000 positions, so that a run is a whole item, and V above 0, so that what the products
    cut off adds up.  Many columns: two steps' 48 products cut off up to 2^-23 of their sum each, of which there are
    118, each added with 2^-24: (48 + 59) 2^-23.  (All 235 steps in one sum would lose about 235 x 24 x 2^-24 / 2,
    1.7e-4.)  Few: the 16 positions of three products lose 3 x 2^-23, and 470 sums are added to a warp's, each
    rounded by 2^-24 at most, evenly to both sides: sqrt(470 / 3) 2^-24 as a norm, of which six times that are allowed."""
    n, hd, G = 30000, 64, 8
    pool, table = make([n] * 19, G, hd, seed=48)
    pool.abs_()
    q = randn((19, rows, 4 * G, hd), 49, F32, 1.5)
    out = paged.attention(q, pool, table, i32([n] * 19))
    most = (48 + 59) * 2.0 ** -23 if rows > 1 else 3 * 2.0 ** -23 + 6 * math.sqrt(470 / 3) * 2.0 ** -24
    for i in (0, 18):
        k, v = R.rows_of(pool, table, i, n)
        want = torch.cat([R.attend(q[i, :, 4 * g:4 * g + 4], k[:, g:g + 1], v[:, g:g + 1], n - rows, 1 / math.sqrt(hd))[0] for g in range(G)], 1)
        assert float((out[i].double() - want).norm() / want.norm()) < most

"""The operators on the 16-bit paged cache on the GPU, against tests/_paged.py."""
import math

import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300 import paged
from tests import _paged as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(shape, seed, dtype=F32, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=gen(seed)) * scale).to(dtype)


def make(lengths, G, hd, seed=0, width=None, spread=1.0):
    """A pool whose sequences hold random rows, everything else NaN."""
    table, n_pages = R.table_for(lengths, seed=seed, width=width)
    pool = torch.full((n_pages, 2, G, R.PAGE, hd), math.nan, dtype=BF, device="cuda")
    for i, n in enumerate(lengths):
        if n:
            R.put(pool, table, i, 0, randn((n, G, hd), 100 * seed + 2 * i, scale=spread), randn((n, G, hd), 100 * seed + 2 * i + 1, scale=spread))
    return pool, table


def check(q, pool, table, lengths, n_new=None, scale=None, mass=None, decay=1.0, out=None, left_out=None):
    """One call, with its log-sum-exp, held to the 64-bit attention and its bounds; with `mass`
    (float32, the values before the call) the masses too.  Returns what the call returned."""
    n, rows, H, hd = q.shape
    G = pool.shape[2]
    sc = 1 / math.sqrt(hd) if scale is None else scale
    got_mass = None if mass is None else mass.clone()
    nn_dev = None if n_new is None else i32(n_new)
    status = i32([0])
    ret, lse = paged.attention(q, pool, table, i32(lengths), n_new=nn_dev, scale=scale, out=out, return_lse=True, mass=got_mass,
                               decay=decay, status=status)
    assert ret.dtype == q.dtype and ret.shape == q.shape and status.item() == 0
    for i, ln in enumerate(lengths):
        nn = rows if n_new is None else n_new[i]
        lo = max(0, nn - ln)                   # rows before it have a negative position
        for r0, r1 in ((0, lo), (nn, rows)):   # padding
            assert not ret[i, r0:r1].any() and bool((lse[i, r0:r1] == -math.inf).all())
        if mass is not None and (nn == 0 or ln == 0):
            assert torch.equal(got_mass[i], mass[i])
        if nn <= lo:
            continue
        k, v = R.rows_of(pool, table, i, ln)
        want, wl, w, A, D = R.attend(q[i, lo:nn], k, v, max(0, ln - nn), sc, None if left_out is None else left_out[i])
        inner, half, lse_off = R.bounds(A, D, wl, ln, hd, q.dtype)
        inner = torch.where(torch.isfinite(inner), inner, 0.0)
        err = (ret[i, lo:nn].double() - want).abs()
        same = torch.isnan(want) & torch.isnan(ret[i, lo:nn]) | (ret[i, lo:nn].double() == want)
        ok = same | (err <= inner + (want.abs() + inner) * half)
        assert bool(ok.all()), (i, int((~ok).sum()), float(err[~ok].max()) if (~ok).any() else 0)
        gl = lse[i, lo:nn].double()
        ok = (gl == wl) | (torch.isnan(gl) & torch.isnan(wl)) | ((gl - wl).abs() <= lse_off)
        assert bool(ok.all()), (i, float((gl - wl).abs().max()))
        if mass is not None:
            new, off = R.mass_step(mass[i, :, :ln].double(), w, D, wl, ln, hd, nn, decay, H // G)
            err = (got_mass[i, :, :ln].double() - new).abs()
            assert bool((err <= off).all()), (i, float((err - off).max()))
            assert torch.equal(got_mass[i, :, ln:], mass[i, :, ln:])
    return ret, lse, got_mass


def masses(table, G, seed=5):
    """Masses whose values behind the ends are NaN, which nothing may touch or use."""
    return torch.exp(2 * randn((table.shape[0], G, R.PAGE * table.shape[1]), seed))


# ---------------------------------------------------------------- store

@pytest.mark.parametrize("hd,G,dtype", [(128, 4, BF), (128, 1, F32), (64, 2, F32), (64, 3, BF)])
@pytest.mark.parametrize("lengths,rows,n_new", [([1], 1, None), ([130, 64], 3, None), ([5, 0, 257, 40], 7, [7, 0, 3, 7]), ([300], 300, None)])
def test_store_writes_the_rows_and_nothing_else(gpu_lib, hd, G, dtype, lengths, rows, n_new):
    table, n_pages = R.table_for(lengths, seed=len(lengths))
    pool = randn((n_pages, 2, G, R.PAGE, hd), 1, BF)
    n = len(lengths)
    wide = randn((n, rows, 3 * G * hd), 2, dtype)        # slices of a wider tensor, as they come from a fused projection
    k, v = wide[..., G * hd:2 * G * hd].unflatten(-1, (G, hd)), wide[..., 2 * G * hd:].unflatten(-1, (G, hd))
    want = pool.clone()
    for i, ln in enumerate(lengths):
        nn = rows if n_new is None else n_new[i]
        lo = max(0, nn - ln)
        if nn > lo:
            R.put(want, table, i, max(0, ln - nn), k[i, lo:nn], v[i, lo:nn])
    status = i32([0])
    paged.store(pool, table, i32(lengths), k, v, n_new=None if n_new is None else i32(n_new), status=status)
    assert torch.equal(pool, want) and status.item() == 0


def test_store_of_special_values(gpu_lib):
    x = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 1e-45, 3.4e38, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8] + [1.0] * 55, device="cuda")
    table, n_pages = R.table_for([1])
    pool = torch.zeros((n_pages, 2, 1, R.PAGE, 64), dtype=BF, device="cuda")
    paged.store(pool, table, i32([1]), x.view(1, 1, 1, 64), -x.view(1, 1, 1, 64))
    page = int(table[0, 0])
    for j, y in ((0, x), (1, -x)):
        got, want = pool[page, j, 0, 0], y.to(BF)
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


# ---------------------------------------------------------------- attention

HEADS = [(16, 4, 128), (4, 2, 64), (8, 1, 128), (4, 4, 64), (10, 2, 128), (3, 1, 64)]


@pytest.mark.parametrize("H,G,hd", HEADS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("lengths", [[1], [127], [128], [129, 1, 64], [2049], [256, 700, 0, 1500, 33]])
def test_single_rows(gpu_lib, H, G, hd, dtype, weigh, lengths):
    pool, table = make(lengths, G, hd, seed=1)
    q = randn((len(lengths), 1, H, hd), 3, dtype, 1.5)
    check(q, pool, table, lengths, mass=masses(table, G) if weigh else None, decay=0.5)


@pytest.mark.parametrize("H,G,hd", HEADS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lengths,rows,n_new", [
    ([5], 5, None), ([300, 4, 129], 4, [4, 4, 1]), ([200, 3, 0, 64], 9, [9, 9, 2, 0]), ([513], 20, None), ([140, 700], 33, [33, 17]),
    ([70], 70, None), ([1000], 100, None), ([900, 40, 300], 130, [130, 130, 1]), ([1300], 257, None)])
def test_several_rows(gpu_lib, H, G, hd, dtype, lengths, rows, n_new):
    pool, table = make(lengths, G, hd, seed=2)
    q = randn((len(lengths), rows, H, hd), 4, dtype, 1.5)
    check(q, pool, table, lengths, n_new=n_new, mass=masses(table, G), decay=0.9)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 6, 300])
def test_many_sequences(gpu_lib, dtype, rows):
    lengths = [(37 * i * i) % 900 + 1 for i in range(40)]
    pool, table = make(lengths, 4, 128, seed=3)
    q = randn((40, rows, 16, 128), 6, dtype)
    check(q, pool, table, lengths, n_new=[(7 * i) % (rows + 1) for i in range(40)], mass=masses(table, 4))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,n", [(1, 33000), (3, 20001), (64, 9000), (1024, 8022)])
def test_long_contexts(gpu_lib, dtype, rows, n):
    pool, table = make([n], 2, 128, seed=4)
    q = randn((1, rows, 4, 128), 7, dtype, 1.5)
    check(q, pool, table, [n], mass=masses(table, 2))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 5, 40, 200])
@pytest.mark.parametrize("scale,spread", [(4.0, 1.0), (-0.3, 1.0), (0.0, 1.0), (0.1, 30.0)])
def test_scales_and_peaked_scores(gpu_lib, dtype, rows, scale, spread):
    """Scores over hundreds: running maxima move, most weights vanish."""
    lengths = [700, 260]
    pool, table = make(lengths, 2, 64, seed=5, spread=spread)
    q = randn((2, rows, 4, 64), 8, dtype)
    check(q, pool, table, lengths, scale=scale, mass=masses(table, 2))


@pytest.mark.parametrize("rising", [True, False])
@pytest.mark.parametrize("rows", [1, 150])
def test_maxima_that_move_at_every_step(gpu_lib, rising, rows):
    n = 1500
    pool, table = make([n], 2, 64, seed=6)
    k = torch.zeros((n, 2, 64), device="cuda")
    k[:, :, 0] = torch.arange(n, device="cuda").flip(0)[:, None] if not rising else torch.arange(n, device="cuda")[:, None]
    R.put(pool, table, 0, 0, k, randn((n, 2, 64), 3))
    q = torch.zeros((1, rows, 4, 64), dtype=BF, device="cuda")
    q[..., 0] = 1.0
    check(q, pool, table, [n], scale=0.25, mass=masses(table, 2))


# ---------------------------------------------------------------- masks

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("rows", [3, 6, 12, 100, 300])
def test_what_a_row_does_not_see_never_shows(gpu_lib, dtype, bad, rows):
    """Values that are no numbers in the K of one of the call's own positions and the V of another:
    rows before them are whole, rows behind them are as the formula has them."""
    n, G, H, hd = 700, 2, 8, 128
    pool, table = make([n], G, hd, seed=7)
    page = table[0].long()
    pv, pk = n - rows // 2, n - 1
    pool[page[pv // 128], 1, 0, pv % 128, 5] = bad
    pool[page[pv // 128], 1, 1, pv % 128, 77] = bad
    q = randn((1, rows, H, hd), 9, dtype)
    # (a K that is no number: the last row, which alone sees it, is NaN or has one weight)
    pool[page[pk // 128], 0, 1, pk % 128, 3] = math.nan
    out, lse = paged.attention(q, pool, table, i32([n]), return_lse=True)
    first = n - rows
    k, v = R.rows_of(pool, table, 0, n)
    want, wl, w, A, D = R.attend(q[0, :rows - 1], k.nan_to_num(0.0), v, first, 1 / math.sqrt(hd))
    got = out[0, :rows - 1].double()
    sees = (torch.arange(first, n - 1, device="cuda") >= pv)
    assert bool(torch.isfinite(got[~sees]).all())
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[sees, :H // 2, 5] = True
    hit[sees, H // 2:, 77] = True
    assert bool(torch.isfinite(got[~hit]).all())
    if math.isnan(bad):
        assert bool(got[hit].isnan().all())
    else:
        assert bool((got[hit] == bad).all())
    inner, half, off = R.bounds(A, D, wl, n, hd, dtype)
    fine = torch.isfinite(want)
    assert bool(((got - want).abs()[fine] <= (inner + (want.abs() + inner) * half)[fine]).all())
    assert bool(((lse[0, :rows - 1].double() - wl).abs() <= off).all())
    assert bool(out[0, -1, H // 2:].isnan().all()) and bool(torch.isfinite(out[0, -1, :H // 2]).any())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 20, 150])
def test_rows_that_see_nothing(gpu_lib, dtype, rows):
    lengths = [0, 3, 200, 0]
    pool, table = make(lengths, 2, 64, seed=8, width=3)
    q = randn((4, rows, 4, 64), 10, dtype)
    check(q, pool, table, lengths, mass=masses(table, 2))
    check(q, pool, table, lengths, n_new=[0, 0, rows, rows], mass=masses(table, 2))
    q[:] = math.nan                            # padding rows may hold anything
    out, lse = paged.attention(q, pool, table, i32(lengths), n_new=i32([0, 0, 0, 0]), return_lse=True)
    assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 9, 150])
def test_keys_of_minus_infinity_and_lowest_values(gpu_lib, dtype, rows):
    """Scores of -inf have no weight; the lowest finite value is a number like any other."""
    n = 300
    pool, table = make([n], 1, 64, seed=9)
    low = torch.finfo(BF).min
    k = torch.zeros((n, 1, 64), device="cuda")
    k[:, :, 0] = randn((n, 1), 4)
    k[5:90, :, 0] = -math.inf
    k[120:130, :, 0] = low
    R.put(pool, table, 0, 0, k, randn((n, 1, 64), 5))
    q = torch.zeros((1, rows, 2, 64), dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    out, lse, _ = check(q, pool, table, [n], scale=1.0, left_out=[(torch.arange(n, device="cuda") >= 5) & (torch.arange(n, device="cuda") < 90)])
    assert bool(torch.isfinite(out).all())
    k[:, :, 0] = -math.inf                     # every score: the row sees positions but none has a weight
    R.put(pool, table, 0, 0, k, randn((n, 1, 64), 5))
    m = masses(table, 1)
    out, lse = paged.attention(q, pool, table, i32([n]), scale=1.0, return_lse=True, mass=m)
    assert not out.any() and bool((lse == -math.inf).all())


# ---------------------------------------------------------------- arguments and status

def test_bad_lengths_and_pages_are_reported_and_left_out(gpu_lib):
    G, hd = 2, 64
    for rows in (1, 40):
        pool, table = make([300, 200], G, hd, seed=10)
        q = randn((2, rows, 4, hd), 11, BF)
        good = table.clone()
        for bad_page in (-1, pool.shape[0], 2 ** 31 - 1):
            table.copy_(good)
            table[0, 1] = bad_page             # positions 128 .. 255 are not seen
            st, m = i32([0]), masses(table, G)
            m0 = m.clone()
            out, lse = paged.attention(q, pool, table, i32([300, 200]), return_lse=True, mass=m, status=st)
            assert st.item() == L.MK_ERR_DEVICE_INDEX
            gone = torch.zeros(300, dtype=torch.bool, device="cuda")
            gone[128:256] = True
            kv = pool[good[0, :3].long()]
            k, v = (kv[:, j].permute(0, 2, 1, 3).flatten(0, 1)[:300].double() for j in (0, 1))
            want, wl, w, A, D = R.attend(q[0], k, v, 300 - rows, 1 / 8, gone)
            inner, half, off = R.bounds(A, D, wl, 300, hd, BF)
            assert bool(((out[0].double() - want).abs() <= inner + (want.abs() + inner) * half).all())
            new, tol = R.mass_step(m0[0, :, :300].double(), w, D, wl, 300, hd, rows, 1.0, 2)
            assert bool(((m[0, :, :300].double() - new).abs() <= tol).all())
            kk = randn((2, rows, G, hd), 12, BF)
            before, st = pool.clone(), i32([0])
            table[0, 2] = bad_page
            paged.store(pool, table, i32([300, 200]), kk, kk, status=st)
            assert st.item() == L.MK_ERR_DEVICE_INDEX
            R.put(before, good, 1, 200 - rows, kk[1], kk[1])
            assert torch.equal(pool.view(torch.int16), before.view(torch.int16))
        table.copy_(good)
        for lengths, n_new in (([385, 200], None), ([-1, 200], None), ([2 ** 31 - 1, 200], None), ([-2 ** 31, 200], None),
                               ([300, 200], [rows + 1, rows]), ([300, 200], [-1, rows])):
            st = i32([0])
            out = paged.attention(q, pool, table, i32(lengths), n_new=None if n_new is None else i32(n_new), status=st, mass=masses(table, G))
            assert st.item() == L.MK_ERR_DEVICE_INDEX
            one = paged.attention(q[1:], pool, table[1:], i32([200]), status=(s2 := i32([0])))
            assert s2.item() == 0
            assert (out[1].double() - one[0].double()).abs().max() <= 2.0 ** -7 * one.double().abs().max()


def test_strides_out_streams_and_refusals(gpu_lib):
    lengths, G, H, hd = [260, 90], 2, 4, 128
    pool, table = make(lengths, G, hd, seed=11)
    for rows, dtype in ((1, BF), (3, F32), (70, BF)):
        wide = randn((rows, 2, H + 3, hd + 8), 13, dtype)
        q = wide.transpose(0, 1)[:, :, 1:H + 1, 8:] if dtype == BF else wide.transpose(0, 1)[:, :, 1:H + 1, 4:hd + 4]
        want = paged.attention(q.contiguous(), pool, table, i32(lengths))
        out = torch.full((2, rows, H, hd), math.nan, dtype=dtype, device="cuda")
        assert paged.attention(q, pool, table, i32(lengths), out=out) is out
        assert torch.equal(out, want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            again = paged.attention(q, pool, table, i32(lengths))
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(again, want)
    q, m = randn((2, 1, H, hd), 1, BF), masses(table, G)
    ln, ones = i32(lengths), table[:, :1].contiguous()
    bad = [
        lambda: paged.attention(q.half(), pool, table, ln), lambda: paged.attention(q, pool.half(), table, ln),
        lambda: paged.attention(q, pool[:, :1], table, ln), lambda: paged.attention(q, pool, table.long(), ln),
        lambda: paged.attention(q, pool, table, ln[:1]), lambda: paged.attention(q.cpu(), pool, table, ln),
        lambda: paged.attention(q[:1], pool, table, ln), lambda: paged.attention(q[..., ::2], pool, table, ln),
        lambda: paged.attention(q, pool, table, ln, out=q), lambda: paged.attention(q, pool, table, ln, out=q.float()),
        lambda: paged.attention(q, pool, table, ln, mass=m[..., :-128]), lambda: paged.attention(q, pool, table, ln, mass=m.double()),
        lambda: paged.attention(q, pool, table, ln, mass=m.transpose(1, 2).contiguous().transpose(1, 2)),
        lambda: paged.attention(q.clone().requires_grad_(), pool, table, ln),
        lambda: paged.attention(q, pool, table, ln, mass=m.clone().requires_grad_()),
        lambda: paged.attention(q, pool, table, ln, out=pool.view(-1)[:q.numel()].view(q.shape)),
        lambda: paged.attention(q, pool, table, ln, n_new=i32([1])), lambda: paged.attention(q, pool, table, ln, status=i32([0, 0])),
        lambda: paged.store(pool, table, ln, q[:, :, :2], q[:, :, :2].float()), lambda: paged.store(pool, table, ln, q, q),
        lambda: paged.store(pool, table, ln, pool[:2, :1, 0, :2], pool[:2, :1, 0, :2]),
        lambda: paged.evict(pool, table, ln, m, 0), lambda: paged.evict(pool, table, ln, m, 5, recent=6),
        lambda: paged.evict(pool, table, ln, m, 5, recent=-1), lambda: paged.evict(pool, table, ln, m[:1], 5),
        lambda: paged.evict(pool, table, ln, m, 5, new_mass=m[:, :, :128]), lambda: paged.evict(pool, table, ln, m, 5, new_lengths=ln[:1]),
        lambda: paged.evict(pool, table, ln, m, 2 ** 40),
        lambda: paged.evict(pool, ones, ln, m[..., :128].contiguous(), 5, new_lengths=ones.view(-1)),
        lambda: paged.evict(pool, table, ln, m, 5, new_lengths=ln[:1].expand(2)),
    ]
    for f in bad:
        with pytest.raises((ValueError, L.MKError)):
            f()
    for f in (lambda: paged.attention(q, pool, table, ln, scale="x"), lambda: paged.attention(q, pool, table, ln, mass=m, decay=None),
              lambda: paged.evict(pool, table, ln, m, 5.5)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(L.MKError):
        paged.attention(q, pool, table, ln, scale=math.nan)
    with pytest.raises(L.MKError):
        paged.attention(q, pool, table, ln, mass=m, decay=math.inf)
    # heads outside sequences: any strides of rows that lie apart
    big = torch.zeros((G, 2, m.shape[2] + 4), device="cuda")
    mt = big[:, :, :m.shape[2]].transpose(0, 1)
    mt.copy_(m)
    paged.attention(q, pool, table, ln, mass=mt, decay=0.5)
    paged.attention(q, pool, table, ln, mass=m, decay=0.5)
    assert torch.equal(mt, m) and not big[:, :, m.shape[2]:].any()
    none = paged.attention(q[:0], pool, table[:0], ln[:0], return_lse=True, mass=m[:0])
    assert none[0].shape == (0, 1, H, hd) and none[1].shape == (0, 1, H)


def test_same_bits_each_time(gpu_lib):
    lengths = [3000, 500, 129]
    pool, table = make(lengths, 4, 128, seed=12)
    for rows, dtype in ((1, BF), (5, F32), (200, BF), (200, F32)):
        q = randn((3, rows, 16, 128), 14, dtype)
        got = []
        for _ in range(3):
            m = masses(table, 4)
            got.append((*paged.attention(q, pool, table, i32(lengths), return_lse=True, mass=m), m))
        assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(got[0], g))


@pytest.mark.parametrize("dtype,rows,hd", [(F32, 10, 128), (BF, 10, 128), (F32, 9, 64), (BF, 33, 64), (BF, 60, 128), (BF, 6, 128), (BF, 5, 64), (BF, 8, 64)])
def test_blocks_of_several_runs(gpu_lib, dtype, rows, hd):
    """Blocks whose runs follow one another (a run's sums leave through the place of the next one's queries), many times."""
    lengths = [(701 * i) % 3000 + 200 for i in range(60)]
    pool, table = make(lengths, 4, hd, seed=20)
    q = randn((60, rows, 16, hd), 21, dtype, 1.5)
    out, lse, m = check(q, pool, table, lengths, mass=masses(table, 4))
    for _ in range(40):
        mm = masses(table, 4)
        o, l = paged.attention(q, pool, table, i32(lengths), return_lse=True, mass=mm)
        assert torch.equal(o, out) and torch.equal(l, lse) and torch.equal(mm, m)


@pytest.mark.parametrize("hd,rows", [(128, 40), (64, 40), (128, 1)])
def test_long_sums_of_fp32_rows(gpu_lib, hd, rows):
    """One kv head, 30000 positions: runs of many steps.  The products cut off up to 2^-23 of the sum with each of the
    24 that a step of 128 positions has, of which 2 steps go into one sum: 48 2^-23 at most, and each of the 118 sums that
    are then added is rounded by 2^-24 of theirs at most, as norms."""
    n = 30000
    pool, table = make([n] * 6, 1, hd, seed=22)
    q = randn((6, rows, 4, hd), 23, F32, 1.5)
    out = paged.attention(q, pool, table, i32([n] * 6))
    for i in range(6):
        k, v = R.rows_of(pool, table, i, n)
        want, wl, w, A, D = R.attend(q[i], k, v, n - rows, 1 / math.sqrt(hd))
        assert float((out[i].double() - want).norm() / want.norm()) < (48 + 59) * 2.0 ** -23


@pytest.mark.parametrize("dtype,hd,rows", [(BF, 128, 5), (BF, 128, 6), (BF, 64, 6), (BF, 64, 8), (F32, 128, 4), (F32, 64, 4)])
@pytest.mark.parametrize("lengths", [[8], [300, 0, 131], [9000], [2500, 700] * 16, [900] * 70])
def test_the_most_columns_of_each_variant(gpu_lib, dtype, hd, rows, lengths):
    """Few columns, as many as a variant takes and a row less: clusters of all sizes, equal runs, rows that see nothing."""
    pool, table = make(lengths, 4, hd, seed=27)
    q = randn((len(lengths), rows, 16, hd), 28, dtype, 1.5)
    check(q, pool, table, lengths, n_new=[(5 * i) % (rows + 1) if i else rows for i in range(len(lengths))], mass=masses(table, 4), decay=0.7)


@pytest.mark.parametrize("case", [
    *[lambda lib, h=h, c=c: test_several_rows(lib, *h, BF, *c) for h in ((16, 4, 128), (10, 2, 128), (3, 1, 64))
      for c in (([1000], 100, None), ([900, 40, 300], 130, [130, 130, 1]), ([1300], 257, None), ([70], 70, None), ([140, 700], 33, [33, 17]))],
    lambda lib: test_many_sequences(lib, BF, 300), lambda lib: test_long_contexts(lib, BF, 1024, 8022),
    *[lambda lib, s=s: test_scales_and_peaked_scores(lib, BF, 200, *s) for s in ((4.0, 1.0), (-0.3, 1.0), (0.0, 1.0), (0.1, 30.0))],
    *[lambda lib, r=r: test_maxima_that_move_at_every_step(lib, r, 200) for r in (True, False)],
    *[lambda lib, b=b: test_what_a_row_does_not_see_never_shows(lib, BF, b, 300) for b in (math.nan, math.inf, -math.inf)],
    lambda lib: test_rows_that_see_nothing(lib, BF, 200), lambda lib: test_keys_of_minus_infinity_and_lowest_values(lib, BF, 200),
    lambda lib: test_bad_lengths_and_pages_are_reported_and_left_out(lib), lambda lib: test_same_bits_each_time(lib),
    lambda lib: test_blocks_of_several_runs(lib, BF, 60, 128)])
def test_wide_tables(gpu_lib, monkeypatch, case):
    """The width of a table, not the lengths in it, is what a call's work is judged by: wide ones take two tiles of columns a block."""
    plain, sms = R.table_for, torch.cuda.get_device_properties(0).multi_processor_count

    def wide(lengths, spare=2, seed=0, width=None, device="cuda"):
        need = max(-(-n // R.PAGE) for n in lengths)
        return plain(lengths, spare, seed, max(need, width or 0, min(6144, 42 * sms // max(1, len(lengths)))), device)

    monkeypatch.setattr(R, "table_for", wide)
    case(gpu_lib)


def test_kernels_behind_one_another_see_new_lengths(gpu_lib):
    """Store, attention, eviction in place and again, without a pause: each reads what the last one wrote."""
    G, H, hd, keep = 4, 16, 128, 300
    table, n_pages = R.table_for([1024] * 8, seed=24)
    k, v = randn((8, 200, G, hd), 1, BF), randn((8, 200, G, hd), 2, BF)
    q = randn((8, 200, H, hd), 3, BF)

    def go(wait):
        pool, mass, ln, got = paged.new_pool(n_pages, G, hd), paged.new_mass(table, G), i32([0] * 8), []
        for step in range(12):
            rows = 200 if step < 3 else 1 + step % 3
            ln += rows
            paged.store(pool, table, ln, k[:, :rows], v[:, :rows])
            if wait:
                torch.cuda.synchronize()
            out, lse = paged.attention(q[:, :rows], pool, table, ln, mass=mass, decay=0.9, return_lse=True)
            if wait:
                torch.cuda.synchronize()
            kept, _, _ = paged.evict(pool, table, ln, mass, keep, recent=20, new_lengths=ln, new_mass=mass)
            if wait:
                torch.cuda.synchronize()
            got += [out, lse, kept, ln.clone(), mass.clone()]
        return got

    want = go(True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(go(False), want))


def test_calls_on_two_streams_at_once(gpu_lib):
    pool, table = make([2000, 900], 4, 128, seed=25)
    qs = [randn((2, rows, 16, 128), rows, dtype) for rows, dtype in ((1, BF), (60, BF), (60, F32), (3, F32))]
    want = [paged.attention(q, pool, table, i32([2000, 900]), return_lse=True) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[] for _ in qs]
    for _ in range(10):
        for i, (q, s) in enumerate(zip(qs, streams)):
            with torch.cuda.stream(s):
                got[i].append(paged.attention(q, pool, table, i32([2000, 900]), return_lse=True))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for x in g for a, b in zip(x, w))


def test_captured_graphs_follow_their_inputs(gpu_lib):
    """Two graphs over the same tensors, replayed in turn and with other lengths, pages and rows."""
    G, H, hd = 2, 8, 64
    lengths = [900, 300, 1]
    pool, table = make([900, 900, 900], G, hd, seed=13)
    for rows in (1, 40):
        q, ln, nn = randn((3, rows, H, hd), 15, BF), i32(lengths), i32([rows] * 3)
        m = [masses(table, G), masses(table, G, 6)]
        paged.attention(q, pool, table, ln, n_new=nn, mass=m[0].clone())      # (the kernels' first use loads them)
        torch.cuda.synchronize()
        graphs, outs = [], []
        for j in (0, 1):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(paged.attention(q, pool, table, ln, n_new=nn, mass=m[j], return_lse=True))
            graphs.append(g)
        for now, new in (([900, 300, 1], [rows] * 3), ([1, 0, 899], [1, 1, rows]), ([128, 129, 700], [0, 1, rows])):
            ln.copy_(i32(now))
            nn.copy_(i32(new))
            q.copy_(randn(q.shape, sum(now), BF))
            start = [masses(table, G, 20 + j) for j in (0, 1)]
            for j in (0, 1):
                m[j].copy_(start[j])
            for j in (0, 1):
                graphs[j].replay()
            torch.cuda.synchronize()
            for j in (0, 1):
                out, lse, mm = check(q, pool, table, now, n_new=new, mass=start[j])
                assert torch.equal(out, outs[j][0]) and torch.equal(lse, outs[j][1]) and torch.equal(mm, m[j])


def test_offsets_past_32_bits(gpu_lib):
    G, hd, n_pages = 4, 128, 16500                  # 2.16e9 values
    pool = paged.new_pool(n_pages, G, hd)
    table = torch.tensor([[16499, 3, 16498]], dtype=torch.int32, device="cuda")
    k, v = randn((1, 300, G, hd), 1, BF), randn((1, 300, G, hd), 2, BF)
    paged.store(pool, table, i32([300]), k, v)
    assert torch.equal(pool[16498, 0, :, :44], k[0, 256:].transpose(0, 1)) and torch.equal(pool[3, 1], v[0, 128:256].transpose(0, 1))
    for rows in (1, 90):
        check(randn((1, rows, 16, hd), 3, BF), pool, table, [300], mass=masses(table, G))
    m, st = masses(table, G), i32([0])
    before = pool[table[0].long()].clone()
    kept, ln, nm = paged.evict(pool, table, i32([300]), m, 140, recent=3, status=st)
    for g in range(G):
        want = R.evict(m[0, g].cpu(), 300, 140, 3)
        assert kept[0, g].tolist() == want
        for slot, src in enumerate(want):
            if slot != src:
                assert torch.equal(pool[table[0, slot // 128].long(), :, g, slot % 128], before[src // 128, :, g, src % 128])
    assert st.item() == 0 and ln.item() == 140


# ---------------------------------------------------------------- eviction

def check_evict(pool, table, lengths, mass, keep, recent, in_place=False):
    G = pool.shape[2]
    want, st = pool.clone(), i32([0])
    m0, ln = mass.clone(), i32(lengths)
    kept, nl, nm = paged.evict(pool, table, ln, mass, keep, recent=recent, new_lengths=ln if in_place else None,
                               new_mass=mass if in_place else None, status=st)
    assert st.item() == 0 and kept.dtype == torch.int32 and kept.shape == (len(lengths), G, keep)
    assert nl.tolist() == [min(n, keep) for n in lengths]
    if in_place:
        assert nl is ln and nm is mass
    else:
        assert ln.tolist() == lengths and torch.equal(mass.view(torch.int32), m0.view(torch.int32))
    cpu = m0.cpu()
    for i, n in enumerate(lengths):
        for g in range(G):
            src = R.evict(cpu[i, g], n, keep, recent)
            assert kept[i, g].tolist() == src, (i, g)
            dst = [s for s in range(keep) if src[s] >= 0 and src[s] != s]
            if dst:
                a, b = torch.tensor(dst, device="cuda"), torch.tensor([src[s] for s in dst], device="cuda")
                t = table[i].long()
                moved = pool.new_empty(0)
                moved = want[t[b // 128], :, g, b % 128].clone()
                want[t[a // 128], :, g, a % 128] = moved
            m = min(n, keep)
            got = nm[i, g].cpu()
            assert torch.equal(got[:m].view(torch.int32), cpu[i, g][torch.tensor(src[:m], dtype=torch.long)].view(torch.int32))
            rest = cpu[i, g, m:] if in_place else torch.zeros(mass.shape[2] - m)
            assert torch.equal(got[m:].view(torch.int32), rest.view(torch.int32))
    assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
    return kept, nl, nm


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("G,hd", [(4, 128), (1, 64), (3, 64)])
@pytest.mark.parametrize("lengths,keep,recent", [
    ([1], 1, 0), ([2], 1, 1), ([129], 128, 0), ([300, 0, 40, 200], 64, 10), ([300, 64, 65], 64, 64), ([1000], 999, 5), ([700, 512], 300, 0),
    ([2500, 90], 31, 30), ([50, 60], 100, 20)])
def test_evictions(gpu_lib, G, hd, lengths, keep, recent, in_place):
    pool, table = make(lengths, G, hd, seed=14)
    mass = masses(table, G)
    mass[mass < 0.4] = 0.0                       # many ties
    check_evict(pool, table, lengths, mass, keep, recent, in_place)


def test_evictions_into_masses_of_other_strides(gpu_lib):
    pool, table = make([700, 300], 3, 64, seed=26)
    mass = masses(table, 3)
    want = paged.evict(pool.clone(), table, i32([700, 300]), mass, 250, recent=9)
    wide = torch.full((3, 2, mass.shape[2] + 8), 7.0, device="cuda")
    to, ln = wide[:, :, :mass.shape[2]].transpose(0, 1), i32([-1, -1])
    kept, nl, nm = paged.evict(pool, table, i32([700, 300]), mass, 250, recent=9, new_lengths=ln, new_mass=to)
    assert nl is ln and nm is to
    assert torch.equal(kept, want[0]) and torch.equal(nl, want[1]) and torch.equal(nm, want[2])
    assert bool((wide[:, :, mass.shape[2]:] == 7.0).all())


@pytest.mark.parametrize("seqs,n", [(1, 131071), (3, 20000), (40, 4097), (100, 300)])
def test_evictions_of_all_widths(gpu_lib, seqs, n):
    lengths = [n - (i * 7) % min(n, 50) for i in range(seqs)]
    pool, table = make(lengths, 2, 64, seed=15)
    mass = masses(table, 2)
    check_evict(pool, table, lengths, mass, max(1, n // 3), n // 50)
    check_evict(pool, table, lengths, mass, n - 60, 0, in_place=True)


def test_evictions_of_the_largest_table(gpu_lib):
    n = 6144 * 128                                    # more are refused (also by the C call)
    pool, table = paged.new_pool(6144, 1, 64), torch.arange(6143, -1, -1, dtype=torch.int32, device="cuda")[None]
    pool.copy_(randn((6144, 1, 1, 128, 1), 31, BF).expand_as(pool))
    for length in (n, n - 5, 700):
        check_evict(pool, table, [length], masses(table, 1), 5000, 100)
    wider = torch.zeros((1, 6145), dtype=torch.int32, device="cuda")
    with pytest.raises(L.MKError):
        paged.evict(pool, wider, i32([5]), masses(wider, 1), 4)


def test_evictions_of_special_masses(gpu_lib):
    """NaN counts as the largest, -0 ties with 0, negative ones and infinities have their order, all may be equal."""
    n = 600
    pool, table = make([n] * 3, 1, 64, seed=16)
    mass = masses(table, 1)
    mass[0, 0, :n] = 0.0
    mass[0, 0, 1:n:2] = -0.0
    mass[1, 0, :n:3] = math.nan
    mass[1, 0, 1:n:5] = -mass[1, 0, 1:n:5]
    mass[1, 0, 2:n:7] = math.inf
    mass[1, 0, 4:n:7] = -math.inf
    mass[1, 0, 5] = 1e-42
    mass[2, 0, :n] = 1.0
    for keep, recent in ((100, 0), (250, 50), (400, 399), (590, 3)):
        check_evict(pool, table, [n] * 3, mass, keep, recent)


def test_evictions_of_bad_pages_and_lengths(gpu_lib):
    pool, table = make([300, 300], 2, 64, seed=17)
    mass, good = masses(table, 2), table.clone()
    for at, bad in ((0, -1), (2, 10 ** 9)):
        table.copy_(good)
        table[0, at] = bad
        before, st = pool.clone(), i32([0])
        kept, ln, _ = paged.evict(pool, table, i32([300, 300]), mass, 100, recent=10, status=st)
        assert st.item() == L.MK_ERR_DEVICE_INDEX and ln.tolist() == [100, 100]
        p = good[0].long()
        if at == 0:                              # every destination: nothing of the sequence is written
            assert torch.equal(pool[p].view(torch.int16), before[p].view(torch.int16))
        assert kept[0, 0].tolist() == R.evict(mass[0, 0].cpu(), 300, 100, 10)
    table.copy_(good)
    for bad in (-5, 385, 2 ** 31 - 1):
        st = i32([0])
        _, ln, _ = paged.evict(pool, table, i32([bad, 300]), mass, 100, status=st)
        assert st.item() == L.MK_ERR_DEVICE_INDEX and ln.tolist() == [0 if bad < 0 else 100, 100]


def test_a_captured_eviction(gpu_lib):
    pool, table = make([500, 400], 2, 64, seed=18)
    mass, ln = masses(table, 2), i32([500, 400])
    paged.evict(pool.clone(), table, ln, mass, 200, recent=20)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept, nl, nm = paged.evict(pool, table, ln, mass, 200, recent=20)
    for lengths, seed in (([500, 400], 1), ([199, 333], 2), ([0, 512], 3)):
        mass.copy_(masses(table, 2, seed))
        ln.copy_(i32(lengths))
        g.replay()
        torch.cuda.synchronize()
        for i, n in enumerate(lengths):
            for h in range(2):
                assert kept[i, h].tolist() == R.evict(mass[i, h].cpu(), n, 200, 20)
        assert nl.tolist() == [min(n, 200) for n in lengths]


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_cache_on_a_budget(gpu_lib, dtype):
    """A prompt in two chunks, cut to a budget by what its rows gave, then tokens one at a time, each pushing out
    one position of every head: the same attention as over the rows that the kept positions stand for."""
    G, H, hd, keep, recent = 2, 8, 128, 150, 16
    prompt, steps = [400, 170], 12
    table, n_pages = R.table_for([512, 512], seed=19)
    pool = torch.full((n_pages, 2, G, R.PAGE, hd), math.nan, dtype=BF, device="cuda")
    mass = paged.new_mass(table, G)
    ln = i32([0, 0])
    K = [randn((n + steps, G, hd), 30 + i, BF) for i, n in enumerate(prompt)]
    V = [randn((n + steps, G, hd), 40 + i, BF) for i, n in enumerate(prompt)]
    holds = [[[] for _ in range(G)] for _ in prompt]   # what each slot stands for, by the evictions' own words

    def extend(rows, n_new):
        """New rows of both sequences: store, attention with masses, held to the 64-bit attention over what the slots stand for."""
        done = [max(max(h, default=-1) for h in s) + 1 for s in holds]
        k, v = (torch.stack([torch.cat([x[i][d:d + n], x[i].new_zeros(rows - n, G, hd)]) for i, (d, n) in enumerate(zip(done, n_new))])
                for x in (K, V))
        ln.add_(i32(n_new))
        for i, n in enumerate(n_new):
            for h in holds[i]:
                h += range(done[i], done[i] + n)
        paged.store(pool, table, ln, k.to(dtype), v.to(dtype), n_new=i32(n_new))
        q = randn((2, rows, H, hd), sum(done), dtype, 1.5)
        before = mass.clone()
        out, lse = paged.attention(q, pool, table, ln, n_new=i32(n_new), mass=mass, decay=0.98, return_lse=True)
        for i, n in enumerate(n_new):
            for g in range(G):
                if not n:
                    continue
                at = torch.tensor(holds[i][g], device="cuda")
                hs = slice(g * (H // G), (g + 1) * (H // G))
                want, wl, w, A, D = R.attend(q[i, :n, hs], K[i][at, g:g + 1].double(), V[i][at, g:g + 1].double(), len(at) - n, 1 / math.sqrt(hd))
                inner, half, off = R.bounds(A, D, wl, len(at), hd, dtype)
                assert bool(((out[i, :n, hs].double() - want).abs() <= inner + (want.abs() + inner) * half).all())
                assert bool(((lse[i, :n, hs].double() - wl).abs() <= off).all())
                new, tol = R.mass_step(before[i, g:g + 1, :len(at)].double(), w, D, wl, len(at), hd, n, 0.98, H // G)
                assert bool(((mass[i, g:g + 1, :len(at)].double() - new).abs() <= tol).all())

    def evict():
        lengths = ln.tolist()
        before = mass.cpu()
        kept, nl, nm = paged.evict(pool, table, ln, mass, keep, recent=recent, new_lengths=ln, new_mass=mass)
        assert nl is ln and nm is mass
        for i in range(2):
            for g in range(G):
                src = R.evict(before[i, g], lengths[i], keep, recent)
                assert kept[i, g].tolist() == src
                holds[i][g] = [holds[i][g][s] for s in src if s >= 0]

    extend(300, [300, 100])
    extend(100, [100, 70])
    evict()
    for _ in range(steps):
        extend(1, [1, 1])
        evict()
    assert ln.tolist() == [keep, keep]

"""Attention over the 4-bit cache for calls of many query columns (rows x heads of
a kv head), where tiles of 128 columns take over: their edges, outliers among
the cached values, what a row must not do to its neighbours, and calls that
overlap.  The reference and the bounds are those of tests/_kv4.py."""
import math

import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import kv4
from tests import _kv4 as R
from tests.test_gpu_kv4 import BF, F32, check, i32, make, poisoned_pool, rows_of, run, table_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,G,hd,rows", [
    (4, 4, 128, 32), (4, 4, 128, 33), (4, 4, 64, 33), (2, 2, 128, 127), (2, 2, 64, 128), (2, 2, 128, 129),
    (8, 2, 128, 9), (8, 2, 64, 65), (1, 1, 128, 257), (5, 1, 64, 26), (64, 1, 128, 3), (4, 4, 128, 81), (4, 1, 64, 20)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_edges_of_the_column_tiles(gpu_lib, dtype, H, G, hd, rows):
    lengths = [rows, 0, 63, 64, 65, 200, 1]
    n_new = [rows, 0, min(rows, 63), 1, min(rows, 65), rows // 2, min(rows, 3)]
    pool, table = make(lengths, G, hd, seed=21)
    run(rows_of(len(lengths), rows, H, hd, dtype), pool, table, lengths, n_new)
    run(rows_of(len(lengths), rows, H, hd, dtype), pool, table, lengths)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,G,hd,rows,n,length", [
    (4, 1, 128, 40, 1, 9000),      # one item, joined from every block
    (4, 4, 64, 40, 1, 5000),
    (8, 2, 128, 300, 3, 700),      # more items than blocks have time for alone: few parts each
    (2, 2, 64, 130, 40, 70),       # many short ones: several items a block
    (16, 4, 128, 512, 2, 513)])
def test_splits_and_joins(gpu_lib, dtype, H, G, hd, rows, n, length):
    lengths = [max(1, length - 31 * i % length) for i in range(n)]
    pool, table = make(lengths, G, hd, seed=22)
    q = rows_of(n, rows, H, hd, dtype)
    out, _ = run(q, pool, table, lengths)
    for _ in range(20):                    # the same bits whatever the blocks' timing
        assert torch.equal(kv4.attention(q, pool, table, i32(lengths)), out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, None])
@pytest.mark.parametrize("mul", [1e-3, 1.0, 60.0])
def test_flat_negative_and_steep_scores(gpu_lib, dtype, mul, scale):
    lengths = [700, 65]
    pool, table = make(lengths, 2, 128, seed=23)
    run(rows_of(2, 24, 8, 128, dtype, mul=mul), pool, table, lengths, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("spread", [1e-9, 1e4, 1e9])
def test_cache_values_of_any_size(gpu_lib, dtype, spread):
    lengths = [400, 33]
    pool, table = make(lengths, 1, 64, seed=24, spread=spread)
    run(rows_of(2, 45, 2, 64, dtype, mul=1.5 / spread), pool, table, lengths)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("times", [256.0, 4096.0])
def test_outliers_among_the_cached_values(gpu_lib, dtype, hd, times):
    """Some positions' K or V far larger than the rest.  A K operand keeps 2^-21 of the
    largest value of its 64 positions (2^-25 absolutely, where the largest is at least
    7 x 2^-6), a V operand 2^-18 of the sequence's largest for bf16 rows (7 x 2^-9),
    2^-21 for fp32 rows.  So a score may be off by scale sum|q| 2^-21 max|K| more, each weight
    by twice that (numerator and denominator), and the result by so much of max|V| more."""
    n, H, rows = 700, 4, 21
    table, n_pages = table_for([n])
    pool = poisoned_pool(n_pages, 1, hd)
    g = torch.Generator(device="cuda").manual_seed(31)
    k, v = (torch.randn((n, 1, hd), device="cuda", generator=g) for _ in range(2))
    k[5::97] *= times
    v[11::131] *= times
    R.fill(pool, hd, table[0].long()[:-(-n // R.PAGE)], k, v)
    q = rows_of(1, rows, H, hd, dtype)
    out, lse = kv4.attention(q, pool, table, i32([n]), return_lse=True)
    kc, vc = R.cache_values(pool, hd, table[0].long(), n)
    o, l, A, D = R.attend(q[0], kc, vc, n - rows, 1 / math.sqrt(hd))
    inner, half, le = R.bounds(A, D, l, n, hd, dtype, float(vc.abs().max()))
    score = q[0].double().abs().sum(-1) / math.sqrt(hd) * 2.0 ** -21 * float(kc.abs().max())
    # a factor e^x of a weight is off by at most e^x - 1 relatively
    inner = inner + torch.expm1(2 * score)[..., None] * A + (2.0 ** -18 if dtype == BF else 2.0 ** -21) * float(vc.abs().max())
    off = (out[0].double() - o).abs() - (inner * (1 + half) + half * o.abs())
    assert off.max() <= 0, off.max().item()
    assert ((lse[0].double() - l).abs() <= le + score).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_is_not_a_number_stays_with_who_sees_it(gpu_lib, dtype):
    """NaN and infinities in q, and groups of K and V that hold NaN, at positions that some rows see."""
    hd, n, rows, H = 128, 300, 70, 4
    pool, table = make([n, n], 1, hd, seed=25)
    q = rows_of(2, rows, H, hd, dtype)
    lengths = [n, n]
    clean, _ = run(q, pool, table, lengths)
    bad_q = q.clone()
    bad_q[0, 1, 2, 3] = math.nan
    bad_q[1, 60, 0, 0] = math.inf
    out, lse = kv4.attention(bad_q, pool, table, i32(lengths), return_lse=True)
    hit = torch.zeros(out.shape[:3], dtype=torch.bool, device="cuda")
    hit[0, 1, 2] = hit[1, 60, 0] = True
    assert out[hit].isnan().all()
    keep = out.clone()
    keep[hit] = clean[hit]
    _, clean_lse = kv4.attention(q, pool, table, i32(lengths), return_lse=True)
    check(q, pool, table, lengths, None, None, keep, torch.where(hit, clean_lse, lse))
    # V's second group of position 250 is NaN: rows that see it are NaN there and nowhere else
    k, v = (torch.randn((1, 1, 1, hd), device="cuda") for _ in range(2))
    v[..., 70] = math.nan
    bad = pool.clone()
    kv4.store(bad, table, i32([251, 251]), k.expand(2, 1, 1, hd), v.expand(2, 1, 1, hd))
    out = kv4.attention(q, bad, table, i32(lengths))
    first = 250 - (n - rows)               # the first row that sees position 250
    assert out[:, first:, :, 64:].isnan().all() and not out[:, first:, :, :64].isnan().any()
    assert torch.equal(out[:, :first], clean[:, :first])
    # K's: every dimension of the rows that see it
    kv4.store(bad, table, i32([251, 251]), v.expand(2, 1, 1, hd), k.expand(2, 1, 1, hd))
    out = kv4.attention(q, bad, table, i32(lengths))
    assert out[:, first:].isnan().all() and torch.equal(out[:, :first], clean[:, :first])


def test_two_streams_at_once(gpu_lib):
    """Calls of many columns next to each other and to single rows."""
    lengths = [3000, 2500, 10]
    pool, table = make(lengths, 4, 128, seed=26)
    qs = [rows_of(3, (100, 1, 33)[s % 3], 16, 128, BF if s < 6 else F32, seed=s) for s in range(9)]
    ln = i32(lengths)
    want = [kv4.attention(q, pool, table, ln) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [None] * 9
    for j in range(9):
        with torch.cuda.stream(streams[j // 3]):
            got[j] = kv4.attention(qs[j], pool, table, ln)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_captured_call_follows_lengths_and_counts(gpu_lib):
    rows, H, G, hd = 48, 8, 2, 128
    pool, table = make([1500, 900, 300], G, hd, seed=27, width=16)
    q = rows_of(3, rows, H, hd, BF)
    ln, nn = i32([1000, 500, 300]), i32([rows] * 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv4.attention(q, pool, table, ln, n_new=nn)
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out, lse = kv4.attention(q, pool, table, ln, n_new=nn, return_lse=True)
    for lengths, n_new in (([1500, 900, 300], [48, 1, 7]), ([1, 0, 64], [1, 0, 48]), ([20, 129, 300], [48, 48, 0]), ([0, 0, 0], [0, 0, 0])):
        ln.copy_(i32(lengths))
        nn.copy_(i32(n_new))
        out.fill_(9)
        lse.fill_(9)
        gr.replay()
        torch.cuda.synchronize()
        check(q, pool, table, lengths, n_new, None, out, lse)


def test_out_may_not_be_queries_memory(gpu_lib):
    pool, table = make([100], 2, 64, seed=28)
    q = rows_of(1, 40, 4, 64, BF)
    for out in (q, torch.cat([q, q], 1)[:, :40]):
        if out is q:
            with pytest.raises(ValueError, match="out must not overlap q"):
                kv4.attention(q, pool, table, i32([100]), out=out)
        else:
            a = kv4.attention(q, pool, table, i32([100]), out=out)
            assert a is out and torch.equal(a, kv4.attention(q, pool, table, i32([100])))
    both = torch.empty((2, 40, 4, 64), dtype=BF, device="cuda")
    both[:1].copy_(q)
    with pytest.raises(ValueError, match="out must not overlap q"):
        kv4.attention(both[:1], pool, table, i32([100]), out=both.view(-1)[64:64 + q.numel()].view(q.shape))
    kv4.attention(both[:1], pool, table, i32([100]), out=both[1:])
    assert torch.equal(both[1:], kv4.attention(q, pool, table, i32([100])))

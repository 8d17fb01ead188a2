"""The operators on the 16-bit paged cache at the ends of what their arguments may be."""
import math

import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300 import paged
from tests.test_gpu_paged import BF, F32, check, check_evict, gen, i32, make, masses, randn

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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,hd,n", [(40, 128, 400000), (100, 64, 400000), (1, 128, 400000), (3, 64, 60000)])
def test_a_value_that_is_no_number_costs_little(gpu_lib, dtype, rows, hd, n):
    """Runs of whole items, several a block: the search for what of V is no finite number, at a run's end, is over
    long before another warp's wait runs out, which would spoil other sequences.  (All sequences are made of 64 pages;
    four have one of their own with such a value.)"""
    seqs, G, H = 80, 2, 4
    pool = randn((68, 2, G, 128, hd), 51, BF)
    table = torch.randint(0, 64, (seqs, n // 128), dtype=torch.int32, device="cuda", generator=gen(52))
    odd = {0: (0, 9, 5, math.nan), 5: (1, n // 2, 63, math.inf), 37: (0, 70, 0, -math.inf), 79: (1, 0, 17, math.nan)}
    for j, (i, (g, p, d, x)) in enumerate(odd.items()):
        table[i, p // 128] = 64 + j
    q = randn((seqs, rows, H, hd), 53, dtype)
    lengths = i32([n // 128 * 128 - 7 * i for i in range(seqs)])
    want = paged.attention(q, pool, table, lengths)
    for j, (g, p, d, x) in enumerate(odd.values()):
        pool[64 + j, 1, g, p % 128, d] = x
    status = i32([0])
    out = paged.attention(q, pool, table, lengths, status=status)
    assert status.item() == 0
    for i, (g, p, d, x) in odd.items():
        got = out[i, :, 2 * g:2 * g + 2, d]
        assert bool((got.isnan() if math.isnan(x) else got == x).all()), i
        out[i, :, 2 * g:2 * g + 2, d] = want[i, :, 2 * g:2 * g + 2, d]
    assert torch.equal(out, want)


def test_a_refused_eviction_takes_no_memory(gpu_lib):
    pool, table = make([300], 2, 64, seed=54)
    m = masses(table, 2)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(L.MKError):             # two lists of 2^31 - 1
        paged.evict(pool, table, i32([300]), m, 2 ** 31 - 1)
    assert torch.cuda.max_memory_allocated() < before + (1 << 20)


@pytest.mark.parametrize("kind", ["zeros", "equal", "two values"])
@pytest.mark.parametrize("seqs,n,keep,recent", [(8, 4097, 4096, 32), (1, 131071, 32768, 1024), (3, 8448, 2048, 0), (2, 300, 7, 7)])
def test_evictions_of_equal_masses(gpu_lib, kind, seqs, n, keep, recent):
    """Ties for all of a sequence: every position counts in the same place of each pass, and the lowest stay."""
    pool, table = make([n] * seqs, 2, 64, seed=55)
    m = torch.zeros((seqs, 2, table.shape[1] * 128), device="cuda")
    if kind != "zeros":
        m[:] = 0.75
    if kind == "two values":
        m[..., ::3] = 0.5
    check_evict(pool, table, [n] * seqs, m, keep, recent)


@pytest.mark.parametrize("rows", [5, 6])
@pytest.mark.parametrize("width", [None, 700])
def test_drafts_in_tables_of_both_forms(gpu_lib, rows, width):
    """20 and 24 columns of 128 dimensions: the wide kernel where the table stands for much work and no masses follow."""
    lengths = [2500, 0, 700, 4]
    pool, table = make(lengths, 4, 128, seed=56, width=width)
    q = randn((4, rows, 16, 128), 57, BF, 1.5)
    check(q, pool, table, lengths)
    check(q, pool, table, lengths, n_new=[rows, rows, 2, 3], mass=masses(table, 4))


@pytest.mark.parametrize("dtype,rows,weigh", [(BF, 1, False), (F32, 1, True), (BF, 40, False), (BF, 40, True)])
def test_the_largest_table(gpu_lib, dtype, rows, weigh):
    """2^31 - 384 positions of one kv head (masses: a page fewer than without), 64 pages over and over: as good as a softmax over these
    with the logarithm of their counts.  A block's run is 7 (few columns) or 14 million positions, whose sums lose 2^-23 with every addition at
    worst: of the products' as the header says, of the weights' one for each of 16 positions of a lane."""
    hd, pages = 64, 64
    width = 16777214 if weigh else 16777215
    n = width * 128
    pool = randn((pages, 2, 1, 128, hd), 58, BF)
    table = torch.randint(0, pages, (1, width), dtype=torch.int32, device="cuda", generator=gen(59))
    q = randn((1, rows, 1, hd), 60, dtype)
    m = torch.zeros((1, 1, n), device="cuda") if weigh else None
    status = i32([0])
    out, lse = paged.attention(q, pool, table, i32([n]), return_lse=True, mass=m, status=status)
    assert status.item() == 0
    # the last page, of which rows see a part, apart from the counts of the others
    count = torch.bincount(table[0, :-1].long(), minlength=pages).double()
    k, v = (pool[:, j, 0].reshape(-1, hd).double() for j in (0, 1))
    last = table[0, -1].long()
    kk, vv = torch.cat([k, pool[last, 0, 0].double()]), torch.cat([v, pool[last, 1, 0].double()])
    s = torch.einsum("rd,nd->rn", q[0, :, 0].double(), kk) / math.sqrt(hd)
    s[:, :pages * 128] += torch.log(count.repeat_interleave(128))
    sees = torch.arange(128, device="cuda")[None] <= torch.arange(128 - rows, 128, device="cuda")[:, None]
    s[:, pages * 128:] = torch.where(sees, s[:, pages * 128:], -math.inf)
    want, A = torch.softmax(s, -1) @ vv, torch.softmax(s, -1) @ vv.abs()
    off = 2.0 ** -23 * n / 152 / 16
    assert bool(((out[0, :, 0].double() - want).abs() <= off * A + 2.0 ** -8 * (want.abs() + off * A)).all())
    assert bool(((lse[0, :, 0].double() - torch.logsumexp(s, -1)).abs() <= off).all())
    if weigh:
        one = torch.exp(s[:, :pages * 128] - torch.log(count.repeat_interleave(128)) - torch.logsumexp(s, -1)[:, None]).sum(0).view(pages, 128)
        got = m[0, 0].view(width, 128)
        for i in (0, 1, width // 2, width - 2):
            assert bool(((got[i].double() - one[table[0, i].long()]).abs() <= 2 * off * one[table[0, i].long()]).all()), i
        total = sum(float(x.double().sum()) for x in m.view(-1).split(1 << 27))
        assert abs(total - rows) <= off * rows
    del m
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,rows,width", [(BF, 1, 1), (BF, 1, 200), (F32, 1, 200), (BF, 40, 3)])
def test_twenty_thousand_sequences(gpu_lib, dtype, rows, width):
    """Sequences of 0 to 90 positions that share 64 pages: a block each, or many runs a block."""
    seqs, hd, pages = min(20000, 524287 // rows), 64, 64
    pool = randn((pages, 2, 1, 128, hd), 64, BF)
    table = torch.randint(0, pages, (seqs, width), dtype=torch.int32, device="cuda", generator=gen(65))
    lengths = torch.randint(0, 91, (seqs,), dtype=torch.int32, device="cuda", generator=gen(66))
    q = randn((seqs, rows, 1, hd), 67, dtype)
    m = torch.ones((seqs, 1, 128 * width), device="cuda")
    out, lse = paged.attention(q, pool, table, lengths, return_lse=True, mass=m, decay=0.5)
    k, v = (pool[table[:, 0].long(), j, 0].float() for j in (0, 1))
    s = torch.einsum("srd,snd->srn", q[:, :, 0].float(), k).double() / math.sqrt(hd)
    at = torch.arange(128, device="cuda")
    first = lengths.long()[:, None] - rows
    sees = at[None, None] <= (first + torch.arange(rows, device="cuda"))[..., None]
    s = s.masked_fill(~sees, -math.inf)
    want = torch.logsumexp(s, -1)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(lse[..., 0]), fine) and bool(((lse[..., 0].double() - want).abs()[fine] <= 1e-4).all())
    w = torch.where(sees & fine[..., None], torch.exp(s - torch.where(fine, want, 0.0)[..., None]), 0.0)
    o = torch.einsum("srn,snd->srd", w, v.double())
    assert bool(((out[:, :, 0].double() - o).abs() <= 1e-4 * (1 + o.abs()) + (2.0 ** -8 if dtype == BF else 0) * o.abs()).all())
    there = at < lengths[:, None]
    old = torch.where(there, torch.where(at < first, 0.5, 0.0), 1.0)
    assert bool(((m[:, 0, :128].double() - old - w.sum(1)).abs() <= 1e-4 * (1 + w.sum(1))).all()) and bool((m[:, 0, 128:] == 1).all())

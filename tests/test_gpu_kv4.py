"""The 4-bit K/V cache on the GPU: store, load and attention against the format
and the attention restated in 64 bits (tests/_kv4.py)."""
import math

import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300 import kv4
from tests import _kv4 as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def table_for(lengths, spare=2, seed=0, width=None):
    """Scattered pages for the lengths; unused entries are -1, which nothing may follow."""
    need = [-(-n // R.PAGE) for n in lengths]
    perm = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    t = torch.full((len(lengths), width or max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        t[i, :k] = perm[at:at + k]
        at += k
    return t.cuda(), sum(need) + spare


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def poisoned_pool(n_pages, G, hd):
    """Every byte 0xFF: the codes are -7, the scales NaN."""
    return torch.full((n_pages, G, R.record(hd)), 255, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- store and load

@pytest.mark.parametrize("hd,G,dtype", [(128, 4, BF), (128, 1, F32), (64, 2, F32), (64, 3, BF)])
@pytest.mark.parametrize("lengths,rows,n_new", [([1], 1, None), ([130, 64], 3, None), ([5, 0, 257, 40], 7, [7, 0, 3, 8 - 1]),
                                                ([300], 300, None)])
def test_store_writes_the_format_byte_by_byte_and_nothing_else(gpu_lib, hd, G, dtype, lengths, rows, n_new):
    table, n_pages = table_for(lengths, seed=len(lengths))
    pool = torch.randint(0, 256, (n_pages, G, R.record(hd)), dtype=torch.uint8, device="cuda", generator=gen(1))
    n = len(lengths)
    # slices of a wider tensor, as they come from a fused projection
    wide = torch.randn((n, rows, 3 * G * hd), device="cuda", generator=gen(2)).to(dtype)
    k, v = wide[..., G * hd:2 * G * hd].unflatten(-1, (G, hd)), wide[..., 2 * G * hd:].unflatten(-1, (G, hd))
    want = pool.cpu().clone()
    for i, ln in enumerate(lengths):
        nn = rows if n_new is None else n_new[i]
        for r in range(nn):
            p = ln - nn + r
            if p < 0:
                continue
            for kv, x in enumerate((k, v)):
                code, s = R.quantise(x[i, r].cpu())
                for g in range(G):
                    R.put(want, hd, int(table[i, p // R.PAGE]), p % R.PAGE, g, kv, code[g], s[g])
    status = i32([0])
    nn_dev = None if n_new is None else i32(n_new)
    kv4.store(pool, table, i32(lengths), k, v, n_new=nn_dev, status=status)
    assert torch.equal(pool.cpu(), want)
    # and what is loaded is what codes and scales stand for
    for dt in (F32, BF):
        lk, lv = kv4.load(pool, table, i32(lengths), rows, n_new=nn_dev, dtype=dt, status=status)
        for got, x in ((lk, k), (lv, v)):
            code, s = R.quantise(x)
            ref = R.values(code, s)
            for i, ln in enumerate(lengths):
                nn = rows if n_new is None else n_new[i]
                ref[i, nn:] = 0
                ref[i, :max(0, nn - ln)] = 0
            assert torch.equal(got, ref.to(dt))
    assert status.item() == 0


def test_store_of_special_groups(gpu_lib):
    """Zeros, values too small for a scale, ties between two codes, infinities, NaN, the largest finite values."""
    hd = 64
    rows = [torch.zeros(hd), torch.full((hd,), -0.0), torch.full((hd,), 1e-44), torch.full((hd,), 2e-40),
            torch.arange(hd, dtype=torch.float32) % 15 * 0.5 - 3.5,          # scale 0.5 exactly: x / s has halves
            torch.full((hd,), 3.0e38), torch.linspace(-1, 1, hd)]
    rows[4][0] = 3.5
    inf, nan = torch.ones(hd), torch.ones(hd)
    inf[7], nan[9] = math.inf, math.nan
    x = torch.stack(rows + [inf, nan]).view(1, -1, 1, hd).cuda()
    n = x.shape[1]
    table, n_pages = table_for([n])
    pool = poisoned_pool(n_pages, 1, hd)
    kv4.store(pool, table, i32([n]), x, -x)
    for kv, y in ((0, x), (1, -x)):
        code, s = R.quantise(y[0, :, 0].cpu())
        for r in range(n):
            c, sc = R.get(pool.cpu(), hd, int(table[0, 0]), r, 0, kv)
            assert torch.equal(c, code[r]), r
            assert torch.equal(sc.float().isnan(), s[r].float().isnan())
            assert torch.equal(sc.view(torch.int16), s[r].view(torch.int16)) or s[r].isnan().all(), r
    k, _ = kv4.load(pool, table, i32([n]), n, dtype=F32)
    assert k[0, :2].abs().max() == 0 and not k[0, :-2].isnan().any()
    assert k[0, -2:].isnan().all()


# ---------------------------------------------------------------- attention

def make(lengths, G, hd, seed=0, spread=1.0, width=None):
    """A pool whose sequences hold random rows, everything else 0xFF."""
    table, n_pages = table_for(lengths, seed=seed, width=width)
    pool = poisoned_pool(n_pages, G, hd)
    for i, n in enumerate(lengths):
        if n:
            pages = table[i, :-(-n // R.PAGE)].long()
            k, v = (torch.randn((n, G, hd), device="cuda", generator=gen(seed * 100 + 2 * i + j)) * spread for j in (0, 1))
            keep = pool[pages].clone()
            R.fill(pool, hd, pages, k, v)
            # slots past the end stay poisoned
            m = torch.zeros((len(pages), G, R.record(hd)), dtype=torch.bool, device="cuda")
            a, b = hd // 2, hd // R.GROUP * 2
            for slot in range((n - 1) % R.PAGE + 1, R.PAGE):
                t, r = slot // R.TILE, slot % R.TILE
                for o in (0, R.TILE * (a + b)):
                    base = t * R.TILE * 2 * (a + b) + o
                    m[-1, :, base + r * a:base + (r + 1) * a] = True
                    m[-1, :, base + R.TILE * a + r * b:base + R.TILE * a + (r + 1) * b] = True
            pool[pages] = torch.where(m, keep, pool[pages])
    return pool, table


def check(q, pool, table, lengths, n_new=None, scale=None, out=None, lse=None, left_out=None):
    """Compare out and lse with the 64-bit attention within the bounds of tests/_kv4.py."""
    n, rows, H, hd = q.shape
    sc = 1 / math.sqrt(hd) if scale is None else scale
    for i, ln in enumerate(lengths):
        nn = rows if n_new is None else n_new[i]
        lo = max(0, nn - ln)                   # rows before it have a negative position
        for r in list(range(lo)) + list(range(nn, rows)):
            assert out[i, r].abs().max() == 0 and (lse[i, r] == -math.inf).all(), (i, r)
        if lo >= nn:
            continue
        k, v = R.cache_values(pool, hd, table[i, :-(-ln // R.PAGE)].long().clamp(0, pool.shape[0] - 1), ln)
        lost = None if left_out is None else left_out[i]
        o, l, A, D = R.attend(q[i, lo:nn], k if lost is None else k.nan_to_num(), v if lost is None else v.nan_to_num(),
                              ln - nn + lo, sc, lost)
        inner, half, le = R.bounds(A, D, l, ln, hd, q.dtype, float(v.nan_to_num().abs().max()))
        got = out[i, lo:nn].double()
        blind = l == -math.inf                  # rows that see nothing
        assert (got[blind] == 0).all()
        off = (got - o).abs() - (inner * (1 + half) + half * o.abs())
        assert off[~blind].max() <= 0 if (~blind).any() else True, (i, off.max().item())
        gl = lse[i, lo:nn].double()
        assert torch.equal(gl == -math.inf, blind)
        assert ((gl - l).abs()[~blind] <= le[~blind]).all(), (i, (gl - l).abs()[~blind].max().item())


def run(q, pool, table, lengths, n_new=None, scale=None):
    status = i32([0])
    nn = None if n_new is None else i32(n_new)
    out, lse = kv4.attention(q, pool, table, i32(lengths), n_new=nn, scale=scale, return_lse=True, status=status)
    assert status.item() == 0
    check(q, pool, table, lengths, n_new, scale, out, lse)
    # without the log-sum-exp, and again: the same bits
    assert torch.equal(kv4.attention(q, pool, table, i32(lengths), n_new=nn, scale=scale), out)
    return out, lse


def rows_of(n, rows, H, hd, dtype, seed=5, mul=1.5):
    return (torch.randn((n, rows, H, hd), device="cuda", generator=gen(seed)) * mul).to(dtype)


HEADS = [(16, 4, 128), (4, 2, 64), (8, 1, 128), (4, 4, 64), (20, 4, 128), (7, 1, 64), (17, 1, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,G,hd", HEADS)
def test_single_rows_at_every_kind_of_length(gpu_lib, H, G, hd, dtype):
    lengths = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 193, 500, 2049]
    pool, table = make(lengths, G, hd, seed=1)
    run(rows_of(len(lengths), 1, H, hd, dtype), pool, table, lengths)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,G,hd", HEADS)
@pytest.mark.parametrize("rows,lengths,n_new", [
    (2, [1, 2, 64, 65, 300], None),             # the first has a row without a position
    (5, [5, 6, 130, 0, 1029], [5, 0, 3, 2, 5]),
    (17, [17, 200, 3], None),
    (70, [70, 64, 700], [70, 65, 11])])
def test_several_rows_are_causal_and_ragged(gpu_lib, H, G, hd, dtype, rows, lengths, n_new):
    pool, table = make(lengths, G, hd, seed=2)
    run(rows_of(len(lengths), rows, H, hd, dtype), pool, table, lengths, n_new)


@pytest.mark.parametrize("n,length,rows", [(1, 9000, 1), (3, 4000, 1), (40, 700, 1), (200, 90, 1), (1, 5000, 40), (300, 1, 2)])
def test_every_split_of_the_work(gpu_lib, n, length, rows):
    lengths = [max(1, length - 37 * i % length) for i in range(n)]
    pool, table = make(lengths, 4, 128, seed=3)
    run(rows_of(n, rows, 16, 128, BF), pool, table, lengths)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mul,scale", [(1.0, 0.0), (2.0, -0.3), (60.0, None), (1e-3, None), (1.0, 3.0)])
def test_flat_negative_and_steep_scores(gpu_lib, dtype, mul, scale):
    lengths = [700, 65, 1]
    pool, table = make(lengths, 2, 128, seed=4)
    run(rows_of(3, 2, 8, 128, dtype, mul=mul), pool, table, lengths, scale=scale)


@pytest.mark.parametrize("spread", [1e-9, 1e-3, 1e4, 1e9])
def test_cache_values_of_any_size(gpu_lib, spread):
    lengths = [400, 33]
    pool, table = make(lengths, 2, 128, seed=5, spread=spread)
    # scores of about one whatever the cache's size
    run(rows_of(2, 1, 8, 128, F32), pool, table, lengths, scale=1 / (spread * math.sqrt(128)))


def test_rising_and_falling_scores(gpu_lib):
    """The largest score last, first, and in the middle: the running maximum moves at every tile."""
    hd, n = 64, 1500
    table, n_pages = table_for([n] * 3)
    pool = poisoned_pool(n_pages, 1, hd)
    ramp = torch.arange(n, device="cuda").float()
    for i, r in enumerate((ramp, n - ramp, n - (ramp - n / 2).abs())):
        k = torch.zeros((n, 1, hd), device="cuda")
        k[:, 0, 0] = r / 10
        v = torch.randn((n, 1, hd), device="cuda", generator=gen(i))
        R.fill(pool, hd, table[i].long(), k, v)
    q = torch.zeros((3, 1, 2, hd), device="cuda")
    q[..., 0] = 8.0
    for dt in (BF, F32):
        run(q.to(dt), pool, table, [n] * 3)


def test_infinities_and_nan_in_a_row_stay_in_that_row(gpu_lib):
    lengths = [300, 300]
    pool, table = make(lengths, 4, 128, seed=6)
    q = rows_of(2, 3, 16, 128, BF)
    clean = kv4.attention(q, pool, table, i32(lengths))
    q[0, 1, 5, 3] = math.nan
    q[1, 2, 0, 0] = math.inf
    out = kv4.attention(q, pool, table, i32(lengths))
    hit = torch.zeros(out.shape[:3], dtype=torch.bool, device="cuda")
    hit[0, 1, 5] = hit[1, 2, 0] = True
    assert out[hit].isnan().all()
    assert torch.equal(out[~hit], clean[~hit])


def test_bad_lengths_and_pages_are_reported_and_left_out(gpu_lib):
    """The kernels' own checks: a length past the table, a negative one, a count past the rows, and pages outside the pool."""
    hd, lengths = 128, [300, 200, 260]
    pool, table = make(lengths, 2, hd, seed=7, width=3)
    q = rows_of(3, 2, 8, hd, BF)
    good = kv4.attention(q, pool, table, i32(lengths))
    bad = table.clone()
    bad[0, 1] = pool.shape[0]
    bad[2, 0] = -5
    status = i32([0])
    out, lse = kv4.attention(q, pool, bad, i32(lengths), return_lse=True, status=status)
    assert status.item() == L.MK_ERR_DEVICE_INDEX
    lost = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in lengths]
    lost[0][128:256] = True
    lost[2][:128] = True
    check(q, pool, bad, lengths, None, None, out, lse, lost)
    assert torch.equal(out[1], good[1])
    # every page of a sequence outside the pool: its rows see nothing
    status.zero_()
    bad[1] = 1 << 30
    out, lse = kv4.attention(q, pool, bad, i32(lengths), return_lse=True, status=status)
    assert status.item() == L.MK_ERR_DEVICE_INDEX and out[1].abs().max() == 0 and (lse[1] == -math.inf).all()
    # lengths: held to [0, 128 * max_pages]
    status.zero_()
    out = kv4.attention(q, pool, table, i32([300, -4, 260]), status=status)
    assert status.item() == L.MK_ERR_DEVICE_INDEX and out[1].abs().max() == 0 and torch.equal(out[0], good[0])
    status.zero_()
    kv4.attention(q, pool, bad, i32([300, 2 ** 31 - 1, 260]), status=status)
    assert status.item() == L.MK_ERR_DEVICE_INDEX
    # a store leaves such places alone, a load gives zeros
    before = pool.clone()
    k = torch.randn((3, 2, 2, hd), device="cuda", dtype=BF)
    status.zero_()
    kv4.store(pool, torch.full_like(table, 1 << 30), i32(lengths), k, k, status=status)
    assert status.item() == L.MK_ERR_DEVICE_INDEX and torch.equal(pool, before)
    status.zero_()
    lk, lv = kv4.load(pool, torch.full_like(table, -1), i32(lengths), 2, status=status)
    assert status.item() == L.MK_ERR_DEVICE_INDEX and lk.abs().max() == 0 and lv.abs().max() == 0


def test_offsets_past_32_bits(gpu_lib):
    hd, G, n_pages = 128, 4, 66000                      # 4.6 GB
    pool = torch.empty((n_pages, G, R.record(hd)), dtype=torch.uint8, device="cuda")
    length = 300
    table = i32([[n_pages - 1, 5, 62000]])
    pages = table[0].long()
    pool[pages] = 255
    k, v = (torch.randn((1, length, G, hd), device="cuda", generator=gen(j)) for j in (0, 1))
    kv4.store(pool, table, i32([length]), k, v)
    lk, _ = kv4.load(pool, table, i32([length]), length, dtype=F32)
    assert torch.equal(lk, R.values(*R.quantise(k)).float())
    q = rows_of(1, 1, 16, hd, BF)
    out, lse = kv4.attention(q, pool, table, i32([length]), return_lse=True)
    check(q, pool, table, [length], None, None, out, lse)


def test_strided_queries_and_given_out(gpu_lib):
    lengths = [150, 90]
    pool, table = make(lengths, 4, 128, seed=8)
    qkv = torch.randn((2, 3, 16 * 128 + 1024), device="cuda", generator=gen(3)).to(BF)
    q = qkv[..., :2048].unflatten(-1, (16, 128))
    want = kv4.attention(q.contiguous(), pool, table, i32(lengths))
    out = torch.full_like(want, 7.0)
    assert kv4.attention(q, pool, table, i32(lengths), out=out) is out
    assert torch.equal(out, want)
    # heads before rows, and one row shared by all sequences
    t = q.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    assert torch.equal(kv4.attention(t, pool, table, i32(lengths)), want)
    e = q[:1].expand(2, -1, -1, -1)
    assert torch.equal(kv4.attention(e, pool, table, i32(lengths)), kv4.attention(e.contiguous(), pool, table, i32(lengths)))


def test_empty_calls_do_nothing(gpu_lib):
    pool, table = make([10], 2, 64, seed=9)
    none = torch.empty((0, 1), dtype=torch.int32, device="cuda")
    z = i32([]).reshape(0)
    q = torch.empty((0, 1, 4, 64), dtype=BF, device="cuda")
    out, lse = kv4.attention(q, pool, none, z, return_lse=True)
    assert out.shape == q.shape and lse.shape == (0, 1, 4)
    assert kv4.attention(torch.empty((1, 0, 4, 64), dtype=BF, device="cuda"), pool, table, i32([10])).numel() == 0
    before = pool.clone()
    kv4.store(pool, none, z, torch.empty((0, 1, 2, 64), dtype=BF, device="cuda"), torch.empty((0, 1, 2, 64), dtype=BF, device="cuda"))
    k, v = kv4.load(pool, table, i32([10]), 0)
    assert k.shape == (1, 0, 2, 64) and torch.equal(pool, before)


def test_a_sequence_grows_by_store_and_attention(gpu_lib):
    """As a decode loop uses them: prompt stored, then a token at a time, then drafted rows of which some are kept."""
    H, G, hd, n = 16, 4, 128, 3
    prompts = [126, 64, 1]
    table, n_pages = table_for([200] * n)
    pool = poisoned_pool(n_pages, G, hd)
    g = gen(11)
    K = [torch.empty((0, G, hd), device="cuda") for _ in range(n)]
    V = [torch.empty((0, G, hd), device="cuda") for _ in range(n)]
    lengths = [0] * n

    def step(counts, rows):
        k, v = (torch.randn((n, rows, G, hd), device="cuda", generator=g).to(BF) for _ in range(2))
        for i, c in enumerate(counts):
            K[i] = torch.cat([K[i], R.values(*R.quantise(k[i, :c])).float()])
            V[i] = torch.cat([V[i], R.values(*R.quantise(v[i, :c])).float()])
            lengths[i] += c
        kv4.store(pool, table, i32(lengths), k, v, n_new=i32(counts))
        q = rows_of(n, rows, H, hd, BF, seed=lengths[0])
        out, lse = kv4.attention(q, pool, table, i32(lengths), n_new=i32(counts), return_lse=True)
        check(q, pool, table, lengths, counts, None, out, lse)
        for i in range(n):
            ck, cv = R.cache_values(pool, hd, table[i].long(), lengths[i])
            assert torch.equal(ck.float(), K[i]) and torch.equal(cv.float(), V[i])

    step(prompts, max(prompts))
    for _ in range(4):
        step([1] * n, 1)
    step([5, 3, 0], 5)
    for i, back in enumerate((3, 1, 0)):      # rejected drafts: the lengths go back and the places are stored again
        lengths[i] -= back
        K[i], V[i] = K[i][:lengths[i]], V[i][:lengths[i]]
    step([2, 1, 2], 2)


def test_side_stream_and_two_streams_at_once(gpu_lib):
    lengths = [3000, 2500, 10]
    pool, table = make(lengths, 4, 128, seed=10)
    qs = [rows_of(3, 1, 16, 128, BF, seed=s) for s in range(6)]
    ln = i32(lengths)
    want = [kv4.attention(q, pool, table, ln) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None] * 6
    for j in range(6):
        with torch.cuda.stream(streams[j % 2]):
            got[j] = kv4.attention(qs[j], pool, table, ln)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_graphs_follow_the_lengths_and_do_not_share_a_workspace(gpu_lib):
    H, G, hd = 16, 4, 128
    pool, table = make([1500, 900], G, hd, seed=12, width=16)
    q = rows_of(2, 1, H, hd, BF)
    new = torch.randn((2, 1, G, hd), device="cuda", generator=gen(5)).to(BF)
    ln = i32([1000, 500])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            kv4.attention(q, pool, table, ln)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            kv4.store(pool, table, ln, new, new)
            outs.append(kv4.attention(q, pool, table, ln, return_lse=True))
        graphs.append(gr)
    for lengths in ([1000, 500], [1, 129], [1400, 0], [65, 888]):
        ln.copy_(i32(lengths))
        for gr, (out, lse) in zip(graphs, outs):
            out.fill_(9)
            gr.replay()
            torch.cuda.synchronize()
            check(q, pool, table, lengths, None, None, out, lse)
    # both at once on two streams
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    want = outs[0][0].clone()
    for _ in range(5):
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want) and torch.equal(outs[1][0], want)


def test_refusals_of_the_python_layer(gpu_lib):
    pool, table = make([100], 2, 64, seed=13)
    ln, q = i32([100]), rows_of(1, 1, 4, 64, BF)
    ok = dict(q=q, pool=pool, table=table, lengths=ln)
    kv4.attention(**ok)
    for bad in (dict(q=q.half()), dict(q=q[..., ::2]), dict(q=q[0]), dict(q=q.cpu()), dict(q=rows_of(2, 1, 4, 64, BF)),
                dict(q=rows_of(1, 1, 4, 128, BF)), dict(pool=pool.int()), dict(pool=pool[:, :1]), dict(pool=pool.cpu()),
                dict(table=table.long()), dict(table=table[0]), dict(lengths=ln.long()), dict(lengths=i32([1, 2])),
                dict(lengths=ln.cpu()), dict(n_new=i32([1, 1])), dict(status=i32([0, 0])), dict(out=torch.empty_like(q).float()),
                dict(out=torch.empty((1, 1, 4, 128), dtype=BF, device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            kv4.attention(**{**ok, **bad})
    for bad in (dict(q=rows_of(1, 1, 3, 64, BF)), dict(scale=math.inf), dict(scale=math.nan)):
        with pytest.raises(L.MKError) as e:
            kv4.attention(**{**ok, **bad})
        assert e.value.code == L.MK_ERR_INVALID_ARG
    odd = torch.zeros(1 + 4 * 64, dtype=BF, device="cuda")[1:].view(1, 1, 4, 64)
    with pytest.raises(L.MKError):
        kv4.attention(**{**ok, "q": odd})
    k = torch.zeros((1, 1, 2, 64), dtype=BF, device="cuda")
    for a, b in ((k, k.float()), (k[:, :, :1], k[:, :, :1]), (k, k.cpu())):
        with pytest.raises(ValueError):
            kv4.store(pool, table, ln, a, b)
    for kw in (dict(dtype=torch.float16), dict(rows=-1)):
        with pytest.raises(ValueError):
            kv4.load(pool, table, ln, **{"rows": 1, **kw})
    for a in ((0, 2, 64), (4, 0, 64), (4, 2, 96)):
        with pytest.raises(ValueError):
            kv4.new_pool(*a)

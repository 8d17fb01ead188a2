"""Attention over the 4-bit cache where the work is cut into equal runs with partial
results in the workspace (calls that need one): items cut between blocks, several items a
block, every form of the join, and runs longer than the window of addresses that a block
looks up.  The reference and the bounds are those of tests/_kv4.py."""
import pytest
import torch

from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300 import kv4
from tests.test_gpu_kv4 import BF, F32, check, gen, i32, make, rows_of, run

pytestmark = pytest.mark.gpu


def workspace(q, pool, table):
    n, rows, H, hd = q.shape
    c = L.mk_kv4_cache(pool=0x1000, table=0x2000, lengths=0x3000, n_new=None, status=None, n_pages=pool.shape[0],
                       n_kv_heads=pool.shape[1], head_dim=hd, n_seqs=n, max_pages=table.shape[1], rows=rows)
    return L.mk_kv4_attention_bytes(c, H, L.MK_F32 if q.dtype == F32 else L.MK_BF16)


def run_cut(q, pool, table, lengths, n_new=None):
    assert workspace(q, pool, table) > 0          # not the form of one cluster an item
    out, lse = run(q, pool, table, lengths, n_new)
    nn = None if n_new is None else i32(n_new)
    for _ in range(5):                            # the same bits whatever the blocks' timing
        assert torch.equal(kv4.attention(q, pool, table, i32(lengths), n_new=nn), out)
    return out, lse


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,G,hd", [(16, 4, 128), (4, 2, 64), (5, 1, 64), (7, 1, 128)])
def test_one_long_sequence_is_joined_from_many_blocks(gpu_lib, dtype, H, G, hd):
    for n in (21001, 40959):                      # above and below the number of parts that picks the join's form
        pool, table = make([n], G, hd, seed=31)
        run_cut(rows_of(1, 1, H, hd, dtype), pool, table, [n])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,G,hd", [(16, 4, 128), (4, 2, 64), (5, 1, 64)])
def test_many_ragged_sequences_with_empty_ones_between(gpu_lib, dtype, H, G, hd):
    """More entries than one scan of a warp takes, several items a block, lengths of 0 and 1 among long ones."""
    lengths = [[3000 - 41 * i, 0, 1, 129][i % 4] for i in range(70)]
    pool, table = make(lengths, G, hd, seed=32, width=128)
    run_cut(rows_of(70, 1, H, hd, dtype), pool, table, lengths)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,H,G,hd", [
    (2, 16, 4, 128), (3, 16, 4, 128), (5, 16, 4, 128), (8, 16, 4, 128),   # 8, 12, 20, 32 columns
    (4, 4, 2, 64), (3, 5, 1, 64), (2, 7, 1, 128), (20, 4, 1, 64)])        # gqa of 2, 5 and 7; 80 columns
def test_drafted_rows(gpu_lib, dtype, rows, H, G, hd):
    lengths = [8022 - 501 * i for i in range(15)] + [2]
    n_new = [(rows, 0, 1, rows - 1)[i % 4] for i in range(16)]
    pool, table = make(lengths, G, hd, seed=33, width=256)
    q = rows_of(16, rows, H, hd, dtype)
    run_cut(q, pool, table, lengths, n_new)
    run_cut(q, pool, table, lengths)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,rows", [(2, 1), (3, 1), (1, 9), (1, 10), (95, 1), (96, 1), (64, 8), (65, 8)])
def test_both_sides_of_the_joins_thresholds(gpu_lib, dtype, n, rows):
    """16 heads on 4: 32 to 8320 columns, of few items and many, so that a column is a block's work with more or
    fewer parts in flight, or a warp's in groups of 8 and 16."""
    lengths = [1500 - 13 * i for i in range(n)]
    pool, table = make(lengths, 4, 128, seed=34, width=256)
    run_cut(rows_of(n, rows, 16, 128, dtype), pool, table, lengths)


def test_a_short_sequence_in_a_wide_table(gpu_lib):
    """The table's width, not the lengths, sizes the work: what a captured decode graph has."""
    for lengths in ([1], [129, 5, 0], [64] * 9):
        for dtype in (BF, F32):
            pool, table = make(lengths, 4, 128, seed=35, width=1024)
            run_cut(rows_of(len(lengths), 1, 16, 128, dtype), pool, table, lengths)


@pytest.mark.parametrize("dtype,rows,gqa,G,n", [
    (BF, 1, 4, 4, 20500), (F32, 3, 4, 4, 10500),   # narrow: more than 64 and 128 steps a block
    (BF, 33, 1, 4, 20500), (F32, 81, 1, 4, 10500)])  # tiles of 128 columns: more than 256 steps a block
def test_runs_longer_than_the_address_window(gpu_lib, dtype, rows, gqa, G, n):
    hd, seqs = 64, 64
    lengths = [n - 7 * i for i in range(seqs)]
    pool, table = make(lengths, G, hd, seed=36)
    q = rows_of(seqs, rows, gqa * G, hd, dtype)
    assert workspace(q, pool, table) > 0
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    wide = rows > 8
    step = 128 if dtype == BF and not wide else 64
    blocks = sms * ({(BF, 0): 4, (F32, 0): 2, (BF, 1): 2, (F32, 1): 1}[dtype, int(wide)])
    per = sum(-(-x // step) for x in lengths) * G / blocks
    assert per > (256 if wide else 64), per
    out, lse = kv4.attention(q, pool, table, i32(lengths), return_lse=True)
    check(q, pool, table, lengths, None, None, out, lse)


def test_two_streams_at_once(gpu_lib):
    lengths = [21000, 2500, 10]
    pool, table = make(lengths, 4, 128, seed=37)
    qs = [rows_of(3, 1 + s % 2 * 4, 16, 128, BF if s < 4 else F32, seed=s) for s in range(8)]
    assert all(workspace(q, pool, table) > 0 for q in qs)
    ln = i32(lengths)
    want = [kv4.attention(q, pool, table, ln) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [None] * 8
        for j in range(8):
            with torch.cuda.stream(streams[j % 2]):
                got[j] = kv4.attention(qs[j], pool, table, ln)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,rows", [(BF, 1), (F32, 1), (BF, 5), (BF, 12), (F32, 24)])
def test_captured_graphs_with_a_workspace_each(gpu_lib, dtype, rows):
    """Two graphs of the same call, with partial results, follow the lengths and run at once."""
    H, G, hd = 16, 4, 128
    pool, table = make([3000, 2100, 1700], G, hd, seed=38, width=256)
    qs = [rows_of(3, rows, H, hd, dtype, seed=s) for s in (1, 2)]
    assert workspace(qs[0], pool, table) > 0
    ln = i32([1000, 500, 90])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv4.attention(qs[0], pool, table, ln)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for q in qs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(kv4.attention(q, pool, table, ln, return_lse=True))
        graphs.append(gr)
    for lengths in ([1000, 500, 90], [3000, 2100, 1700], [1, 0, 129], [rows, 2100, 64]):
        ln.copy_(i32(lengths))
        for gr, q, (out, lse) in zip(graphs, qs, outs):
            out.fill_(9)
            gr.replay()
            torch.cuda.synchronize()
            check(q, pool, table, lengths, None, None, out, lse)
    ln.copy_(i32([3000, 2100, 1700]))
    for gr in graphs:
        gr.replay()
    torch.cuda.synchronize()
    want = [out.clone() for out, _ in outs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, w) for (out, _), w in zip(outs, want))

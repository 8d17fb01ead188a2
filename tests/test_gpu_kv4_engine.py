"""The engine on a 4-bit cache, and forks, truncation and compaction of the
page pool (both cache formats), on the tiny model."""
import numpy as np
import pytest
import torch

import synth
from oracle import Oracle
from oracle.model import ContiguousKV
from synth import prompts as SP
from synth import weights as SW
from moe_decode_megakernel_persistent_gb300 import _lib as L
from moe_decode_megakernel_persistent_gb300.engine import Batcher, Engine, PrefixCache, Request
from tests import _kv4 as R
from tests import _parity as PR

pytestmark = pytest.mark.gpu

TINY = synth.CONFIGS[1].model


class QuantisedKV(ContiguousKV):
    """The oracle's cache in 4 bits: k and v keep the bf16 rows (what a write
    gets), read() gives what the codes stand for."""

    def __init__(self, *a):
        super().__init__(*a)
        self.q = {}

    def read(self, layer, T):
        out = []
        for name, rows in (("k", self.k[layer]), ("v", self.v[layer])):
            done = self.q.get((name, layer))
            if done is None or len(done) < T:
                n = 0 if done is None else len(done)
                new = R.values(*R.quantise(torch.from_numpy(rows[n:T]))).numpy()
                done = self.q[(name, layer)] = new if n == 0 else np.concatenate([done, new])
            out.append(done[:T])
        return out

    def quantised(self, start, n):
        both = [np.stack([self.read(l, start + n)[j][start:] for l in range(len(self.k))]) for j in (0, 1)]
        return torch.from_numpy(np.stack(both, axis=2))


class Oracle4(Oracle):
    def new_kv(self):
        return QuantisedKV(self.m.n_layers, self.m.n_kv_heads, self.m.head_dim)


@pytest.fixture(scope="module")
def tiny():
    out = {}

    def get(wdtype):
        if wdtype not in out:
            m = TINY.with_(wdtype=wdtype)
            out[wdtype] = (m, SW.model_torch(m, "cuda"))
        return out[wdtype]
    return get


def check_written(rep, eng, kv, seq, start, n, tag):
    """What the GPU's rows read back as is near what the oracle's do: a row in the wrong place is off wholesale,
    a value next to the border of two codes by a seventh of its group's largest."""
    g = eng.kv_read(seq, start, n).double().cpu().numpy()
    w = kv.quantised(start, n).numpy()
    e = PR.rel_l2(g.reshape(g.shape[0] * n, -1), w.reshape(g.shape[0] * n, -1))
    if (e > PR.KV_TOL).any():
        rep.failures.append(f"{tag}: kv rel_l2 {e.max():.3e}")


@pytest.mark.parametrize("wdtype", ["f32", "bf16", "int4"])
@pytest.mark.parametrize("prompt_len,own", [(200, 16), (300, 40), (130, 1), (1000, 5)])
def test_steps_over_the_4_bit_cache_match_the_oracle(gpu_lib, tiny, wdtype, prompt_len, own):
    """The cache holds the oracle's rows (mk_kv_write rounds them to the same
    codes); the last `own` prompt rows run on the GPU (one launch per layer up
    to 16 rows, the GEMM path for 40), then three decode steps, each compared
    layer by layer."""
    m, w = tiny(wdtype)
    orc, rep, tol = Oracle4(m, PR.host_fetch(m, w)), PR.Report(), 2e-2
    prompt = SP.prompt_tokens(m.seed, m.vocab, prompt_len, seq=3)
    kv = orc.new_kv()
    tok_o, tr_o = orc.prefill(kv, prompt)
    eng = Engine(m, w, n_pages=16, max_ctx=1100, max_seqs=4, kv_dtype="int4")
    eng.enable_trace(16)
    first = prompt_len - own
    eng.kv_write(2, 0, PR.oracle_kv(kv, 0, first))
    out = eng.prefill(2, torch.from_numpy(prompt[first:]).cuda(), start_pos=first)
    eng.sync()
    rows = own - ((own - 1) // 16) * 16
    tg = eng.split_trace(rows)
    PR.compare_trace(rep, m, tg, tr_o, slice(0, rows), slice(prompt_len - rows, prompt_len), tol, "prefill", "p")
    PR.check_token(rep, int(out.item()), tok_o, float(tr_o["top2_margin"][-1]), "prefill", "p")
    check_written(rep, eng, kv, 2, first, own, "prefill")
    eng.kv_write(2, first, PR.oracle_kv(kv, first, own))
    cur, tin, tout = tok_o, torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    for i in range(3):
        pos = prompt_len + i
        nxt, tr_o = orc.decode(kv, cur, pos)
        tin.fill_(cur)
        eng.decode_step([2], tin, [pos], tout)
        eng.sync()
        PR.compare_trace(rep, m, eng.split_trace(1), tr_o, slice(0, 1), slice(0, 1), tol, f"step {i}", i)
        PR.check_token(rep, int(tout.item()), nxt, float(tr_o["top2_margin"][-1]), f"step {i}", i)
        check_written(rep, eng, kv, 2, pos, 1, f"step {i}")
        eng.kv_write(2, pos, PR.oracle_kv(kv, pos, 1))
        cur = nxt
    assert not rep.failures, rep
    eng.close()


def test_a_batch_over_the_4_bit_cache_matches_the_oracle_per_sequence(gpu_lib, tiny):
    m, w = tiny("int4")
    lens = [70 + 61 * s for s in range(8)]
    eng = Engine(m, w, n_pages=64, max_ctx=1024, max_seqs=16, kv_dtype="int4")
    orc, rep = Oracle4(m, PR.host_fetch(m, w)), PR.Report()
    ids = [(5 * s + 3) % 16 for s in range(8)]
    nxt, kvs = [], []
    for s, n in enumerate(lens):
        kv = orc.new_kv()
        t, _ = orc.prefill(kv, SP.prompt_tokens(m.seed, m.vocab, n, seq=s))
        eng.kv_write(ids[s], 0, PR.oracle_kv(kv, 0, n))
        nxt.append(t)
        kvs.append(kv)
    toks = torch.tensor(nxt, dtype=torch.int32, device="cuda")
    eng.enable_trace(8)
    eng.decode_step(ids, toks, lens, toks)
    eng.sync()
    tr = eng.split_trace(8)
    for s, n in enumerate(lens):
        _, tro = orc.decode(kvs[s], nxt[s], n)
        PR.compare_trace(rep, m, tr, tro, slice(s, s + 1), slice(0, 1), 2e-2, f"seq {s}", seq=s)
        PR.check_token(rep, int(toks[s].item()), int(tro["next_token"][-1]), float(tro["top2_margin"][-1]), f"seq {s}", seq=s)
        check_written(rep, eng, kvs[s], ids[s], n, 1, f"seq {s}")
    assert not rep.failures, rep
    eng.close()


def test_the_4_bit_engine_gives_the_same_bits_again_and_split(gpu_lib, tiny):
    m, w = tiny("int4")
    p = torch.from_numpy(SP.prompt_tokens(m.seed, m.vocab, 150, seq=1)).cuda()
    got = []
    for flags in (0, 0, L.MK_DBG_SPLIT):
        eng = Engine(m, w, n_pages=8, max_ctx=512, max_seqs=2, kv_dtype="int4")
        if flags:
            L.mk_set_debug(eng.ctx, flags)
        tok = eng.prefill(0, p)
        toks = [int(tok.item())]
        for i in range(6):
            eng.decode_step([0], tok, [150 + i], tok)
            toks.append(int(tok.item()))
        eng.sync()
        got.append((toks, eng.kv_read(0, 0, 156).clone()))
        eng.close()
    for toks, kv in got[1:]:
        assert toks == got[0][0] and torch.equal(kv.view(torch.int16), got[0][1].view(torch.int16))


def test_batcher_and_prefix_cache_run_on_the_4_bit_engine(gpu_lib, tiny):
    m, w = tiny("int4")
    eng = Engine(m, w, n_pages=32, max_ctx=1024, max_seqs=12, max_batch=4, kv_dtype="int4")
    ps = [torch.from_numpy(SP.prompt_tokens(m.seed, m.vocab, n, seq=s)).cuda() for s, n in enumerate((40, 129, 5, 300, 64))]
    out = Batcher(eng).run([Request(seq_id=s, prompt=p, max_new=5, arrival=2 * s) for s, p in enumerate(ps)])
    assert out["launches"] > 0 and eng.info()["free_pages"] == 32
    pc = PrefixCache(eng, capacity=2, whole_pages=False)
    reused = []
    for sid, p in enumerate((ps[3], ps[3], ps[1], ps[3])):
        _, n = pc.prefill(6 + sid, p)
        reused.append(n)
        pc.keep(6 + sid, p.tolist())
    eng.sync()
    assert reused == [0, 299, 0, 299]
    eng.close()


def test_timing_is_refused_on_the_4_bit_cache(gpu_lib, tiny):
    m, w = tiny("int4")
    eng = Engine(m, w, n_pages=4, max_ctx=256, max_seqs=2, kv_dtype="int4")
    eng.enable_timing()
    with pytest.raises(L.MKError) as e:
        eng.prefill(0, torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert e.value.code == L.MK_ERR_UNSUPPORTED and eng.seq_length(0) == -1 and eng.info()["free_pages"] == 4
    with pytest.raises(ValueError):
        Engine(m, w, n_pages=4, kv_dtype="int3")
    with pytest.raises(L.MKError) as e:
        L.mk_kv_alloc_fmt(eng.ctx, 4, L.MK_BF16)
    assert e.value.code == L.MK_ERR_STATE
    eng.close()


def test_kv_transfers_of_the_4_bit_cache(gpu_lib, tiny):
    m, w = tiny("int4")
    eng = Engine(m, w, n_pages=80, max_ctx=10000, max_seqs=3, kv_dtype="int4")
    g = torch.Generator(device="cuda").manual_seed(7)
    n = 9000                                       # more pages than one launch enters
    kv = torch.randn((m.n_layers, n, 2, m.n_kv_heads, m.head_dim), generator=g, device="cuda").to(torch.bfloat16)
    eng.kv_write(1, 0, kv)
    want = R.values(*R.quantise(kv)).to(torch.bfloat16)
    assert torch.equal(eng.kv_read(1, 0, n), want) and eng.info()["free_pages"] == 80 - 71
    part = kv[:, 100:300].flip(0).contiguous()
    eng.kv_write(1, 50, part)
    want[:, 50:250] = R.values(*R.quantise(part)).to(torch.bfloat16)
    assert torch.equal(eng.kv_read(1, 0, n), want)
    assert torch.equal(eng.kv_read(1, 4095, 130), want[:, 4095:4225])
    with pytest.raises(L.MKError) as e:
        eng.kv_write(2, 0, kv[:, :1300].contiguous())      # 11 pages, 9 left
    assert e.value.code == L.MK_ERR_NO_PAGES and eng.seq_length(2) == -1 and eng.info()["free_pages"] == 9
    eng.sync()
    eng.close()


# ---------------------------------------------------------------- pages of the pool

def rows(m, n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((m.n_layers, n, 2, m.n_kv_heads, m.head_dim), generator=g, device="cuda").to(torch.bfloat16)


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_fork_at_any_length(gpu_lib, tiny, fmt):
    m, w = tiny("int4")
    eng = Engine(m, w, n_pages=7, max_ctx=1024, max_seqs=6, kv_dtype=fmt)
    eng.kv_write(0, 0, rows(m, 300, 1))                      # 3 pages
    src = eng.kv_read(0, 0, 300)
    for seq, n, taken in ((1, 200, 1), (2, 256, 0), (3, 1, 1), (4, 300, 1)):
        free = eng.info()["free_pages"]
        eng.fork_at(0, seq, n)
        assert eng.info()["free_pages"] == free - taken and eng.seq_length(seq) == n
        assert same(eng.kv_read(seq, 0, n), src[:, :n].contiguous())
    with pytest.raises(L.MKError) as e:                      # no page for another tail
        eng.kv_write(2, 256, rows(m, 1, 9))                  # takes the last one
        eng.fork_at(0, 5, 130)
    assert e.value.code == L.MK_ERR_NO_PAGES and eng.seq_length(5) == -1
    # each goes on in its own last page
    eng.kv_write(1, 200, rows(m, 40, 2))
    eng.kv_write(0, 260, rows(m, 40, 3))
    eng.kv_write(4, 290, rows(m, 30, 4))
    assert same(eng.kv_read(1, 0, 200), src[:, :200].contiguous()) and same(eng.kv_read(0, 0, 260), src[:, :260].contiguous())
    assert same(eng.kv_read(4, 0, 290), src[:, :290].contiguous()) and same(eng.kv_read(3, 0, 1), src[:, :1].contiguous())
    for args, code in (((0, 1, 5), L.MK_ERR_STATE), ((5, 1, 5), L.MK_ERR_STATE), ((0, 0, 5), L.MK_ERR_INVALID_ARG),
                       ((0, 5, 0), L.MK_ERR_INVALID_ARG), ((0, 5, 301), L.MK_ERR_INVALID_ARG), ((0, 6, 5), L.MK_ERR_INVALID_ARG),
                       ((-1, 5, 5), L.MK_ERR_INVALID_ARG)):
        with pytest.raises(L.MKError) as e:
            eng.fork_at(*args)
        assert e.value.code == code, args
    for s in range(5):
        eng.release(s)
    assert eng.info()["free_pages"] == 7
    eng.sync()
    eng.close()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_truncate_gives_pages_back_and_never_writes_a_shared_one(gpu_lib, tiny, fmt):
    m, w = tiny("int4")
    eng = Engine(m, w, n_pages=6, max_ctx=1024, max_seqs=4, kv_dtype=fmt)
    eng.kv_write(0, 0, rows(m, 500, 1))                      # 4 pages
    a = eng.kv_read(0, 0, 500)
    eng.truncate(0, 500)
    eng.truncate(0, 385)
    assert eng.seq_length(0) == 385 and eng.info()["free_pages"] == 2
    eng.truncate(0, 384)
    assert eng.seq_length(0) == 384 and eng.info()["free_pages"] == 3
    assert same(eng.kv_read(0, 0, 384), a[:, :384].contiguous())
    eng.fork(0, 1, 256)                                      # shares pages 0 and 1
    eng.truncate(1, 200)                                     # its last page becomes its own
    assert eng.info()["free_pages"] == 2
    eng.kv_write(1, 200, rows(m, 56, 2))
    assert same(eng.kv_read(0, 0, 384), a[:, :384].contiguous()) and same(eng.kv_read(1, 0, 200), a[:, :200].contiguous())
    eng.fork(0, 2, 256)
    eng.truncate(0, 129)                                     # the source's page is shared with 2
    assert eng.info()["free_pages"] == 2                     # one freed, one taken
    eng.kv_write(0, 129, rows(m, 10, 3))
    assert same(eng.kv_read(2, 0, 256), a[:, :256].contiguous())
    eng.fork(2, 3, 128)
    eng.kv_write(3, 128, rows(m, 200, 4))
    assert eng.info()["free_pages"] == 0
    with pytest.raises(L.MKError) as e:                      # page 0 is shared and there is no page to copy it to
        eng.truncate(2, 100)
    assert e.value.code == L.MK_ERR_NO_PAGES and eng.seq_length(2) == 256
    eng.truncate(2, 128)
    assert eng.seq_length(2) == 128 and eng.info()["free_pages"] == 1
    for args, code in (((2, 129), L.MK_ERR_INVALID_ARG), ((2, 0), L.MK_ERR_INVALID_ARG), ((9, 1), L.MK_ERR_INVALID_ARG)):
        with pytest.raises(L.MKError) as e:
            eng.truncate(*args)
        assert e.value.code == code
    eng.release(1)
    with pytest.raises(L.MKError) as e:
        eng.truncate(1, 1)
    assert e.value.code == L.MK_ERR_STATE
    eng.sync()
    eng.close()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_truncated_drafts_leave_no_trace(gpu_lib, tiny, fmt):
    """Five tokens run past position 130 and are taken back: what follows has the bits of a run without them."""
    m, w = tiny("int4")
    p = torch.from_numpy(SP.prompt_tokens(m.seed, m.vocab, 126, seq=2)).cuda()
    runs = []
    for drafts in (False, True):
        eng = Engine(m, w, n_pages=4, max_ctx=512, max_seqs=2, kv_dtype=fmt)
        tok = eng.prefill(0, p)
        if drafts:
            first = tok.clone()
            eng.prefill(0, p[:5], start_pos=126)             # crosses into the second page
            assert eng.info()["free_pages"] == 2
            eng.truncate(0, 126)
            assert eng.info()["free_pages"] == 3
            tok = first
        got = []
        for i in range(6):
            eng.decode_step([0], tok, [126 + i], tok)
            got.append(int(tok.item()))
        eng.sync()
        runs.append((got, eng.kv_read(0, 0, 132).clone()))
        eng.close()
    assert runs[0][0] == runs[1][0] and same(runs[0][1], runs[1][1])


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_compaction_moves_pages_and_nothing_else(gpu_lib, tiny, fmt):
    m, w = tiny("int4")
    eng = Engine(m, w, n_pages=200, max_ctx=16384, max_seqs=12, kv_dtype=fmt)
    assert eng.compact() == 0
    lens = [300, 128, 1, 4000, 129, 7000, 40, 900]           # 3, 1, 1, 32, 2, 55, 1, 8 pages
    for s, n in enumerate(lens):
        eng.kv_write(s, 0, rows(m, n, s))
    eng.fork(3, 8, 2560)                                     # 20 shared pages
    eng.fork_at(5, 9, 6000)                                  # 46 shared, one copied
    held = {s: n for s, n in enumerate(lens)}
    held.update({8: 2560, 9: 6000})
    for s in (0, 2, 3, 7):
        eng.release(s)
        del held[s]
    before = {s: eng.kv_read(s, 0, n).clone() for s, n in held.items()}
    free = eng.info()["free_pages"]
    live = 200 - free
    assert live == 1 + 2 + 55 + 1 + 20 + 1
    # live pages numbered live or above move: pages were handed out from 0 up
    moved = eng.compact()
    assert 0 < moved <= live and eng.info()["free_pages"] == free
    assert eng.compact() == 0                                # there is nothing left to move
    for s, n in held.items():
        assert same(eng.kv_read(s, 0, n), before[s]), s
    # the pages handed out next are the free ones
    eng.kv_write(0, 0, rows(m, free * 128, 50))
    assert eng.info()["free_pages"] == 0
    for s, n in held.items():
        assert same(eng.kv_read(s, 0, n), before[s]), s
    for s in list(held) + [0]:
        eng.release(s)
    assert eng.info()["free_pages"] == 200
    eng.sync()
    eng.close()


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_decoding_goes_on_over_compacted_pages(gpu_lib, tiny, fmt):
    m, w = tiny("int4")
    ps = [torch.from_numpy(SP.prompt_tokens(m.seed, m.vocab, n, seq=n)).cuda() for n in (260, 140, 300)]
    runs = []
    for compact in (False, True):
        eng = Engine(m, w, n_pages=12, max_ctx=1024, max_seqs=4, kv_dtype=fmt)
        toks = [eng.prefill(s, p) for s, p in enumerate(ps)]
        eng.release(0)
        t = torch.cat(toks[1:])
        got = []
        for i in range(4):
            if compact and i == 1:
                assert eng.compact() == 3                    # pages 3..7 are in use, five of them: 5, 6 and 7 move
            eng.decode_step([1, 2], t, [140 + i, 300 + i], t)
            got.append(t.tolist())
        eng.sync()
        runs.append((got, [eng.kv_read(s, 0, n).clone() for s, n in ((1, 144), (2, 304))]))
        eng.close()
    assert runs[0][0] == runs[1][0] and all(same(a, b) for a, b in zip(runs[0][1], runs[1][1]))


def test_prefix_cache_to_the_token(gpu_lib, tiny):
    """Turns A, A, B, A with whole_pages=False: 599 of 600 tokens are reused, and every turn's token is the oracle's
    wherever its top-2 margin is clear."""
    m, w = tiny("int4")
    orc, ref, rep, reused = Oracle(m, PR.host_fetch(m, w)), {}, PR.Report(), []
    for name, seq in (("A", 0), ("B", 1)):
        p = SP.prompt_tokens(m.seed, m.vocab, 600, seq=seq)
        tok, tr = orc.prefill(orc.new_kv(), p)
        ref[name] = (torch.from_numpy(p).cuda(), tok, float(tr["top2_margin"][-1]))
    eng = Engine(m, w, n_pages=32, max_ctx=1024, max_seqs=8)
    pc = PrefixCache(eng, capacity=2, whole_pages=False)
    for sid, name in enumerate("AABA"):
        p, tok, margin = ref[name]
        out, n = pc.prefill(sid, p)
        eng.sync()
        reused.append(n)
        PR.check_token(rep, int(out.item()), tok, margin, f"turn {sid}", seq=sid)
        pc.keep(sid, p.tolist())
    assert reused == [0, 599, 0, 599] and not rep.failures, (reused, rep)
    eng.close()

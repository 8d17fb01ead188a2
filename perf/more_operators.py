"""Workloads of the operators on a paged 16-bit key/value cache: the store,
causal attention of single rows and of chunks of new rows, the same with the
weights that each cached position receives added up, and the eviction of the
positions that received least.

A pool of one layer is a bfloat16 tensor [n_pages, 2, n_kv_heads, 128, head_dim]
(K, then V): one layer of the engine's cache.  Sequence i of a call holds
lengths[i] positions, position p in slot p % 128 of page table[i][p // 128]; its
new rows (all `rows` of the call, or n_new[i] of them) are the last ones of these.

mass is float32 [n_seqs, n_kv_heads, positions]: what a position has received, the
softmax weights summed over the rows and the query heads of its kv head.  A call
with it sets mass[p] = decay * mass[p] + (what the call's rows give p), where the
call's own new positions start from nothing.  Eviction leaves `keep` positions of
each (sequence, kv head): the last `recent` and the heaviest others, ties to the
lower position.  Those below `keep` stay; the rest move into the free slots below
it, in order.

With `own` false, `run` computes the plain form; with `own` true, it calls the
framework.
"""
import math

import torch

own = False

PAGE = 128          # positions of a page


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of one sequence: the context of the shortest Flint workload, where latency counts
        dict(name="attend step 2049", op="attend", seqs=1, lo=2049, hi=2049, rows=1, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # 64 clients up to 16384 tokens: the largest decode step
        dict(name="attend 64 clients", op="attend", seqs=64, lo=4096, hi=16384, rows=1, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # a prompt chunk against the cache it extends
        dict(name="attend chunk 1024", op="attend", seqs=1, lo=8022, hi=8022, rows=1024, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # the chunks of three prompts of different lengths in one call, in the engine's fp32 rows
        dict(name="attend chunks f32", op="attend", seqs=3, lo=700, hi=2049, rows=641, heads=16, kv_heads=4, dim=128,
             dtype="f32", ragged=True),
        # the decode step of the 16-client workload, prompts of 256 to 8192 tokens, with the weights kept
        dict(name="weigh 16 clients", op="weigh", seqs=16, lo=256, hi=8448, rows=1, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False, decay=1.0),
        # a prompt chunk whose weights say what of the prompt to keep
        dict(name="weigh chunk 1024", op="weigh", seqs=1, lo=8022, hi=8022, rows=1024, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False, decay=1.0),
        # drafted tokens of a ragged batch in the tiny fp32 model's heads, older weights fading
        dict(name="weigh drafts f32", op="weigh", seqs=7, lo=1, hi=3000, rows=5, heads=4, kv_heads=2, dim=64,
             dtype="f32", ragged=True, decay=0.95),
        # the prompts of 16 clients cut to a budget after their prefill
        dict(name="evict 16 prompts", op="evict", seqs=16, lo=256, hi=8448, keep=2048, recent=64, kv_heads=4, dim=128),
        # one long context cut to a quarter
        dict(name="evict long 131071", op="evict", seqs=1, lo=131071, hi=131071, keep=32768, recent=1024, kv_heads=4, dim=128),
        # 64 clients at their budget: the token of the step pushes out one position of each head
        dict(name="evict step 64", op="evict", seqs=64, lo=4097, hi=4097, keep=4096, recent=32, kv_heads=4, dim=128),
        # the new K/V of one decode step of 16 sequences
        dict(name="store step 16", op="store", seqs=16, lo=256, hi=8448, rows=1, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # the K/V of a whole prompt chunk, as the engine has them
        dict(name="store chunk 4096 f32", op="store", seqs=1, lo=8022, hi=8022, rows=4096, heads=16, kv_heads=4, dim=128,
             dtype="f32", ragged=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(16, 4, 128), (16, 4, 128), (4, 2, 64), (8, 1, 128), (4, 4, 64), (20, 4, 128)]


def draw(rng):
    op = rng.choice(["attend"] * 4 + ["weigh"] * 4 + ["evict"] * 3 + ["store"] * 2)
    heads, kv_heads, dim = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    seqs = _log(rng, 1, 64)
    if op == "store":
        rows = _log(rng, 1, max(1, 4096 // seqs))
        hi = rows + _log(rng, 1, 4000)
        return dict(op=op, seqs=seqs, lo=rng.randint(max(1, rows // 2), hi), hi=hi, rows=rows, heads=heads, kv_heads=kv_heads,
                    dim=dim, dtype=dtype, ragged=rng.random() < 0.5)
    hi = _log(rng, 1, min(131072, 600000 // seqs))
    lo = _log(rng, 1, hi)
    if op == "evict":
        keep = _log(rng, 1, hi)
        return dict(op=op, seqs=seqs, lo=lo, hi=hi, keep=keep, recent=rng.choice([0, rng.randint(0, keep), keep // 8]),
                    kv_heads=kv_heads, dim=dim)
    rows = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 1024)])
    rows = max(1, min(rows, 5_000_000 // (seqs * hi)))
    c = dict(op=op, seqs=seqs, lo=lo, hi=hi, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
             ragged=rows > 1 and rng.random() < 0.5)
    if op == "weigh":
        c["decay"] = rng.choice([1.0, 0.9, 0.5])
    return c


# ---------------------------------------------------------------- inputs

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lengths(c):
    """Lengths from the case alone, so that work() knows them: spread over [lo, hi], the ends among them."""
    n = c["seqs"]
    if n == 1:
        return [c["hi"]]
    return [c["lo"] + (c["hi"] - c["lo"]) * ((i * 7919) % n) // (n - 1) for i in range(n)]


def _n_new(c):
    """New rows of each sequence: all of the call's, or in a ragged batch 0 .. rows of them."""
    return [c["rows"] - (i * 3 % (c["rows"] + 1) if c["ragged"] else 0) for i in range(c["seqs"])]


def _table(lengths, extra, gen, dev):
    """Pages of every sequence in scattered order; entries past a sequence's pages are 0."""
    need = [-(-x // PAGE) for x in lengths]
    perm = torch.randperm(sum(need) + extra, generator=gen, device=dev).to(torch.int32)
    rows = torch.zeros(len(lengths), max(1, max(need)), dtype=torch.int32, device=dev)
    at = 0
    for i, k in enumerate(need):
        rows[i, :k] = perm[at:at + k]
        at += k
    return rows, sum(need) + extra


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    lengths = _lengths(c)
    table, n_pages = _table(lengths, 3, gen, dev)
    g, d = c["kv_heads"], c["dim"]
    # every slot holds values, those behind a sequence's end too, as in a page that held another
    pool = torch.empty((n_pages, 2, g, PAGE, d), dtype=torch.bfloat16, device=dev)
    pool.normal_(generator=gen)
    s = dict(op=c["op"], pool=pool, table=table, lengths=torch.tensor(lengths, dtype=torch.int32, device=dev))
    positions = table.shape[1] * PAGE
    if c["op"] in ("weigh", "evict"):
        # what has been received so far: over some binades, a part of the positions nothing (ties)
        m = torch.exp(2 * torch.randn((c["seqs"], g, positions), device=dev, generator=gen))
        s["mass"] = torch.where(torch.rand(m.shape, device=dev, generator=gen) < 0.1, 0.0, m)
    if c["op"] == "evict":
        s.update(keep=c["keep"], recent=c["recent"])
        return s
    s["rows"] = c["rows"]
    s["n_new"] = torch.tensor(_n_new(c), dtype=torch.int32, device=dev) if c["ragged"] else None
    h = c["heads"]
    if c["op"] == "store":
        # k and v are slices of the projection's output, as they come from it
        qkv = torch.randn((c["seqs"], c["rows"], (h + 2 * g) * d), device=dev, generator=gen).to(DT[c["dtype"]])
        s["k"] = qkv[..., h * d:(h + g) * d].unflatten(-1, (g, d))
        s["v"] = qkv[..., (h + g) * d:].unflatten(-1, (g, d))
        return s
    s["q"] = (torch.randn((c["seqs"], c["rows"], h, d), device=dev, generator=gen) * 1.5).to(DT[c["dtype"]])
    s["decay"] = c.get("decay")
    return s


# ---------------------------------------------------------------- plain forms

def _new(s):
    return s["n_new"].long() if s["n_new"] is not None else torch.full_like(s["lengths"], s["rows"]).long()


def _limits(s):
    """How many positions row r of sequence i sees: [seqs, rows], 0 for rows that see nothing."""
    r = torch.arange(s["rows"], device=s["lengths"].device)
    n = _new(s)[:, None]
    return torch.where(r < n, (s["lengths"].long()[:, None] - n + r + 1).clamp(min=0), 0)


def _plain_attend(s):
    q = s["q"]
    kv = s["pool"][s["table"].long()].permute(2, 0, 3, 1, 4, 5).flatten(3, 4).float()   # [2, S, G, T, d]
    S, R, H, d = q.shape
    G, T = kv.shape[2], kv.shape[3]
    at = torch.arange(T, device=q.device)
    length = s["lengths"].long()[:, None]
    qg = q.float().view(S, R, G, H // G, d).permute(0, 2, 3, 1, 4).reshape(S, G, -1, d)
    x = torch.matmul(qg, kv[0].transpose(-1, -2)).unflatten(2, (H // G, R)) / math.sqrt(d)
    x = x.masked_fill(at >= _limits(s)[:, None, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    # what a masked place holds is no number to rely on
    v = torch.where((at < length)[:, None, :, None], kv[1], 0.0)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (H // G, R)).permute(0, 3, 1, 2, 4).reshape(S, R, H, d).to(q.dtype)
    lse = (m + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(S, R, H)
    if s["op"] == "attend":
        return out, lse
    mass, n = s["mass"], _new(s)[:, None]
    old = torch.where((at < length - n)[:, None], s["decay"] * mass, 0.0)
    there = ((at < length) & (n > 0))[:, None]
    mass.copy_(torch.where(there, old + p.sum((2, 3)), mass))
    return out, lse, mass


def _plain_evict(s):
    mass, length, keep = s["mass"], s["lengths"].long()[:, None, None], s["keep"]
    S, G, T = mass.shape
    at = torch.arange(T, device=mass.device).expand(S, G, T)
    # the last `recent` first, then by mass, then what lies behind the end
    worth = torch.where(at >= length - s["recent"], math.inf, mass)
    worth = torch.where(at < length, worth, -math.inf)
    order = worth.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, at)
    kept = (rank < keep) & (at < length)
    free = (at < keep) & (at < length) & ~kept
    late = kept & (at >= keep)
    # slots below keep: those that stay, and for the i-th free one the i-th late position
    source = torch.full((S, G, keep + 1), -1, dtype=torch.int64, device=mass.device)
    nth = torch.full((S, G, keep + 1), -1, dtype=torch.int64, device=mass.device)
    nth.scatter_(-1, torch.where(late, late.long().cumsum(-1) - 1, keep), at)
    head = at[..., :min(keep, T)]
    source[..., :head.shape[-1]] = torch.where(kept[..., :keep], head, torch.where(
        free[..., :keep], nth.gather(-1, (free.long().cumsum(-1) - 1)[..., :keep].clamp(min=0)), -1))
    source = source[..., :keep]
    i, g, slot = torch.nonzero((source >= 0) & (source != torch.arange(keep, device=mass.device)), as_tuple=True)
    src = source[i, g, slot]
    table, pool = s["table"].long(), s["pool"]
    pool[table[i, slot // PAGE], :, g, slot % PAGE] = pool[table[i, src // PAGE], :, g, src % PAGE]
    held = mass.gather(-1, source[..., :T].clamp(min=0))
    new = torch.zeros_like(mass)
    new[..., :held.shape[-1]] = torch.where(source[..., :T] >= 0, held, 0.0)
    return pool, source.to(torch.int32), s["lengths"].clamp(max=keep), new


def _plain_store(s):
    r = torch.arange(s["rows"], device=s["lengths"].device)
    n = _new(s)[:, None]
    p = s["lengths"].long()[:, None] - n + r
    i, row = torch.nonzero((r < n) & (p >= 0), as_tuple=True)
    p = p[i, row]
    page = s["table"].long()[i, p // PAGE]
    for j, x in enumerate((s["k"], s["v"])):
        s["pool"][page, j, :, p % PAGE] = x[i, row].to(torch.bfloat16)
    return s["pool"]


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        from moe_decode_megakernel_persistent_gb300 import paged
        if s["op"] == "store":
            paged.store(s["pool"], s["table"], s["lengths"], s["k"], s["v"], n_new=s["n_new"])
            return s["pool"]
        if s["op"] == "evict":
            kept, lengths, mass = paged.evict(s["pool"], s["table"], s["lengths"], s["mass"], s["keep"], recent=s["recent"])
            return s["pool"], kept, lengths, mass
        if s["op"] == "weigh":
            out, lse = paged.attention(s["q"], s["pool"], s["table"], s["lengths"], n_new=s["n_new"], return_lse=True,
                                       mass=s["mass"], decay=s["decay"])
            return out, lse, s["mass"]
        return paged.attention(s["q"], s["pool"], s["table"], s["lengths"], n_new=s["n_new"], return_lse=True)
    if s["op"] == "store":
        return _plain_store(s)
    return _plain_evict(s) if s["op"] == "evict" else _plain_attend(s)


def work(case):
    c = case
    lengths, g, d = _lengths(c), c["kv_heads"], c["dim"]
    held = 2 * d * 2                                           # bytes of one position of one kv head
    if c["op"] == "evict":
        # the masses are alike for all positions, so that the kept ones are spread over them
        keep, recent, moves = c["keep"], c["recent"], 0.0
        for n in lengths:
            if n > keep:
                late = min(recent, n - keep)
                moves += g * (late + (keep - recent) * (n - keep - late) / max(1, n - recent))
        positions = -(-max(lengths) // PAGE) * PAGE
        return {"bytes": 2 * moves * held + g * 4 * sum(lengths) + c["seqs"] * g * 4 * (keep + positions), "flops": g * sum(lengths)}
    size = 2 if c["dtype"] == "bf16" else 4
    new = _n_new(c)
    if c["op"] == "store":
        n = sum(min(a, b) for a, b in zip(new, lengths))
        return {"bytes": n * g * (2 * d * size + held), "flops": 2 * n * g * d}
    seen = sum(max(0, b - a + r + 1) for a, b in zip(new, lengths) for r in range(a))
    rows = c["seqs"] * c["rows"] * c["heads"]
    read = sum(b for a, b in zip(new, lengths) if a) * g
    return {"bytes": read * (held + (8 if c["op"] == "weigh" else 0)) + rows * (2 * d * size + 4), "flops": 4 * seen * c["heads"] * d}


# ---------------------------------------------------------------- in 64 bits

def _exact_evict(s, lengths):
    """By its definition: a sequence and head at a time, kept positions sorted by (mass, position)."""
    pool, keep = s["pool"].clone(), s["keep"]
    mass = torch.zeros_like(s["mass"], dtype=torch.float64)
    for i, n in enumerate(lengths):
        pages = s["table"][i].long()
        for g in range(mass.shape[1]):
            m = s["mass"][i, g, :n].double()
            if n <= keep:
                mass[i, g, :n] = m
                continue
            others = n - s["recent"]
            heaviest = torch.argsort(-m[:others], stable=True)[:keep - s["recent"]]
            stays = torch.zeros(n, dtype=torch.bool, device="cuda")
            stays[heaviest] = True
            stays[others:] = True
            src = torch.nonzero(stays[keep:])[:, 0] + keep
            dst = torch.nonzero(~stays[:keep])[:, 0]
            mass[i, g, :keep] = m[:keep]
            mass[i, g, dst] = m[src]
            for j in (0, 1):
                pool[pages[dst // PAGE], j, g, dst % PAGE] = s["pool"][pages[src // PAGE], j, g, src % PAGE]
    return pool.double(), None, None, mass


def exact(case, seed):
    s = prepare(case, seed)
    lengths = _lengths(case)
    if s["op"] == "evict":
        return _exact_evict(s, lengths)
    new = _n_new(case)
    if s["op"] == "store":
        want = s["pool"].double()
        for i, (n, ln) in enumerate(zip(new, lengths)):
            p = torch.arange(max(0, ln - n), ln, device="cuda")
            page = s["table"][i].long()[p // PAGE]
            for j, x in enumerate((s["k"], s["v"])):
                want[page, j, :, p % PAGE] = x[i, n - len(p):n].double()
        return want
    S, R, H, d = s["q"].shape
    G = s["pool"].shape[2]
    out = torch.zeros((S, R, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((S, R, H), -math.inf, dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if s["op"] == "weigh" else None
    for i, (n, ln) in enumerate(zip(new, lengths)):
        pages = s["pool"][s["table"][i, :-(-ln // PAGE)].long()]
        if mass is not None and n:
            mass[i, :, :max(0, ln - n)] *= s["decay"]
            mass[i, :, max(0, ln - n):ln] = 0
        for g in range(G):
            k, v = (pages[:, j, g].reshape(-1, d)[:ln].double() for j in (0, 1))
            hs = slice(g * (H // G), (g + 1) * (H // G))
            for r0 in range(max(0, n - ln), n, 128):
                r1 = min(n, r0 + 128)
                upto = ln - n + r1                               # what the last of these rows sees
                x = torch.einsum("rhd,td->rht", s["q"][i, r0:r1, hs].double(), k[:upto]) / math.sqrt(d)
                sees = torch.arange(upto, device="cuda")[None, :] <= torch.arange(ln - n + r0, upto, device="cuda")[:, None]
                x = torch.where(sees[:, None, :], x, -math.inf)
                lse[i, r0:r1, hs] = torch.logsumexp(x, -1)
                w = torch.softmax(x, -1)
                out[i, r0:r1, hs] = torch.einsum("rht,td->rhd", w, v[:upto])
                if mass is not None:
                    mass[i, g, :upto] += w.sum((0, 1))
    return (out, lse) if mass is None else (out, lse, mass)

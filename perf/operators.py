"""Workloads of the operators on a paged key/value cache: the 4-bit store and
load, attention over the 4-bit cache, and page copies.

A 4-bit pool of one layer is a uint8 tensor [n_pages, n_kv_heads, record] of
pages of 128 positions.  A record is two tiles of 64 positions, a tile
    K codes  uint8    [64][head_dim / 2]
    K scales bfloat16 [64][head_dim / 64]
    V codes, V scales  likewise
Groups of 64 values along head_dim share a scale s = bf16(max|x| / 7); a code
is a sign bit (8) over a magnitude min(7, rint(|x| / s)), the even index in the
low nibble; it stands for +-magnitude * s.  Sequence i of a call holds
lengths[i] positions in the pages table[i]; its new rows (all `rows` of the
call, or n_new[i] of them) are the last ones of these.

With `own` false, `run` computes the plain form; with `own` true, it calls the
framework.
"""
import math

import torch

own = False

PAGE = 128          # positions of a page
TILE = 64           # positions of a tile
GROUP = 64          # values that share a scale


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of one sequence: the context of the shortest Flint workload, where latency counts
        dict(name="attend step 2049", op="attend", seqs=1, lo=2049, hi=2049, rows=1, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # the decode step of the 16-client workload, prompts of 256 to 8192 tokens
        dict(name="attend 16 clients", op="attend", seqs=16, lo=256, hi=8448, rows=1, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # one sequence at a long, odd context
        dict(name="attend long 131071", op="attend", seqs=1, lo=131071, hi=131071, rows=1, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # 64 clients up to 16384 tokens: the largest decode step
        dict(name="attend 64 clients", op="attend", seqs=64, lo=4096, hi=16384, rows=1, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # drafted tokens scored in one call: a ragged batch of up to 5 rows each
        dict(name="attend drafts 16x5", op="attend", seqs=16, lo=100, hi=8022, rows=5, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=True),
        # the tiny fp32 model's heads
        dict(name="attend f32 tiny", op="attend", seqs=7, lo=1, hi=3000, rows=1, heads=4, kv_heads=2, dim=64,
             dtype="f32", ragged=False),
        # a prompt chunk against the cache it extends
        dict(name="attend chunk 1024", op="attend", seqs=1, lo=8022, hi=8022, rows=1024, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # the new K/V of one decode step of 16 sequences
        dict(name="store step 16", op="store", seqs=16, lo=256, hi=8448, rows=1, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # the K/V of a whole prompt chunk
        dict(name="store chunk 4096", op="store", seqs=1, lo=8022, hi=8022, rows=4096, heads=16, kv_heads=4, dim=128,
             dtype="bf16", ragged=False),
        # ragged fp32 rows of the tiny model
        dict(name="store f32 ragged", op="store", seqs=5, lo=200, hi=900, rows=77, heads=4, kv_heads=2, dim=64,
             dtype="f32", ragged=True),
        # a forked sequence's partly filled last page, all 49 layers of the bf16 cache
        dict(name="copy fork bf16", op="copy", layers=49, pages=24, moves=1, kv_heads=4, dim=128, form="bf16"),
        # a compaction that moves 150 pages of the 4-bit cache
        dict(name="copy compact 4-bit", op="copy", layers=49, pages=400, moves=150, kv_heads=4, dim=128, form="4-bit"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(16, 4, 128), (16, 4, 128), (4, 2, 64), (8, 1, 128), (4, 4, 64), (20, 4, 128)]


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "store", "store", "copy"])
    if op == "copy":
        form = rng.choice(["bf16", "4-bit"])
        layers, moves = _log(rng, 1, 49), _log(rng, 1, 150)
        moves = max(1, min(moves, (150 if form == "4-bit" else 40) * 49 // layers // 2))
        return dict(op=op, layers=layers, pages=2 * moves + rng.randint(1, 40), moves=moves, kv_heads=rng.choice([2, 4]),
                    dim=rng.choice([64, 128]), form=form)
    heads, kv_heads, dim = rng.choice(HEADS)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    seqs = _log(rng, 1, 64)
    if op == "store":
        rows = _log(rng, 1, max(1, 4096 // seqs))
        hi = rows + _log(rng, 1, 4000)
        return dict(op=op, seqs=seqs, lo=rng.randint(max(1, rows // 2), hi), hi=hi, rows=rows, heads=heads, kv_heads=kv_heads,
                    dim=dim, dtype=dtype, ragged=rng.random() < 0.5)
    hi = _log(rng, 1, min(131072, 600000 // seqs))
    rows = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 512)])
    rows = max(1, min(rows, 5_000_000 // (seqs * hi)))
    return dict(op=op, seqs=seqs, lo=_log(rng, 1, hi), hi=hi, rows=rows, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                ragged=rows > 1 and rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _record(dim):
    return PAGE * 2 * (dim // 2 + dim // GROUP * 2)


def _lengths(c):
    """Lengths from the case alone, so that work() knows them: spread over [lo, hi], the ends among them."""
    n = c["seqs"]
    if n == 1:
        return [c["hi"]]
    return [c["lo"] + (c["hi"] - c["lo"]) * ((i * 7919) % n) // (n - 1) for i in range(n)]


def _n_new(c):
    """New rows of each sequence: all of the call's, or in a ragged batch 0 .. rows of them."""
    n = [c["rows"] - (i * 3 % (c["rows"] + 1) if c["ragged"] else 0) for i in range(c["seqs"])]
    return n


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
    if c["op"] == "copy":
        if c["form"] == "4-bit":
            pool = torch.randint(0, 256, (c["layers"], c["pages"], c["kv_heads"], _record(c["dim"])), dtype=torch.uint8,
                                 device=dev, generator=gen)
        else:
            pool = torch.randn((c["layers"], c["pages"], 2, c["kv_heads"], PAGE, c["dim"]), dtype=torch.bfloat16, device=dev,
                               generator=gen)
        order = torch.randperm(c["pages"], generator=torch.Generator().manual_seed(seed)).tolist()
        # live pages move into free ones: no page is both
        return dict(op="copy", pool=pool, src=order[:c["moves"]], dst=order[c["moves"]:2 * c["moves"]])
    lengths, n_new = _lengths(c), _n_new(c)
    table, n_pages = _table(lengths, 3, gen, dev)
    s = dict(op=c["op"], table=table, lengths=torch.tensor(lengths, dtype=torch.int32, device=dev), rows=c["rows"],
             n_new=torch.tensor(n_new, dtype=torch.int32, device=dev) if c["ragged"] else None, dim=c["dim"])
    h, g, d = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "store":
        # k and v are slices of the projection's output, as they come from it
        qkv = torch.randn((c["seqs"], c["rows"], (h + 2 * g) * d), device=dev, generator=gen)
        qkv *= torch.rand((c["seqs"], c["rows"], 1), device=dev, generator=gen) * 2 + 0.1
        qkv = qkv.to(DT[c["dtype"]])
        s["k"] = qkv[..., h * d:(h + g) * d].unflatten(-1, (g, d))
        s["v"] = qkv[..., (h + g) * d:].unflatten(-1, (g, d))
        s["pool"] = torch.randint(0, 128, (n_pages, g, _record(d)), dtype=torch.uint8, device=dev, generator=gen)
        return s
    # a cache as the store leaves it, of normal values with a scale of their own
    # for each position (in pieces, so that a large pool takes little memory);
    # what lies behind a sequence's end is filled too, as in a page that held another
    pool = torch.empty((n_pages, g, 2, _record(d) // 2), dtype=torch.uint8, device=dev)
    for at in range(0, n_pages, 512):
        n = min(512, n_pages - at)
        x = torch.randn((n, g, 2, 2, TILE, d), device=dev, generator=gen)
        x *= torch.rand((n, g, 2, 2, TILE, 1), device=dev, generator=gen) + 0.5
        codes, scales = _quantise(x)
        pool[at:at + n] = torch.cat([p for j in (0, 1) for p in (codes[:, :, :, j].flatten(-2),
                                                                 scales[:, :, :, j].flatten(-2).view(torch.uint8))], -1)
    s["pool"] = pool.flatten(-2)
    s["q"] = (torch.randn((c["seqs"], c["rows"], h, d), device=dev, generator=gen) * 1.5).to(DT[c["dtype"]])
    return s


# ---------------------------------------------------------------- plain forms

def _quantise(x):
    """x [..., dim] -> codes uint8 [..., dim / 2] and scales bfloat16 [..., dim / 64]."""
    x = x.float().unflatten(-1, (-1, GROUP))
    s = (x.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16)
    m = torch.where(s > 0, x.abs() / s.float(), torch.zeros_like(x)).round().clamp(max=7).to(torch.uint8)
    code = (m + 8 * ((x < 0) & (m > 0)).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.squeeze(-1)


def _values(codes, scales):
    """The fp32 values that codes and scales stand for, [..., dim]."""
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    v = (nib & 7).float() * (1 - 2 * (nib >> 3).float())
    return (v.unflatten(-1, (-1, GROUP)) * scales.float().unsqueeze(-1)).flatten(-2)


def _parts(tiles, d):
    """The four parts of tiles [..., tile bytes]: K codes, K scales, V codes, V scales, each [..., 64, ...]."""
    a, b = TILE * d // 2, TILE * d // GROUP * 2
    kc, ks, vc, vs = tiles.split((a, b, a, b), -1)
    return (kc.unflatten(-1, (TILE, -1)), ks.contiguous().view(torch.bfloat16).unflatten(-1, (TILE, -1)),
            vc.unflatten(-1, (TILE, -1)), vs.contiguous().view(torch.bfloat16).unflatten(-1, (TILE, -1)))


def _gathered(s):
    """K and V of every sequence's pages in fp32, [seqs, kv heads, positions, dim]."""
    pages = s["pool"][s["table"].long()]                              # [S, P, G, record]
    tiles = pages.unflatten(-1, (2, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)   # [S, G, tiles, bytes]
    kc, ks, vc, vs = _parts(tiles, s["dim"])
    return _values(kc, ks).flatten(2, 3), _values(vc, vs).flatten(2, 3)


def _new(s):
    return s["n_new"].long() if s["n_new"] is not None else torch.full_like(s["lengths"], s["rows"]).long()


def _limits(s):
    """How many positions row r of sequence i sees: [seqs, rows], 0 for rows that see nothing."""
    r = torch.arange(s["rows"], device=s["lengths"].device)
    n = _new(s)[:, None]
    return torch.where(r < n, (s["lengths"].long()[:, None] - n + r + 1).clamp(min=0), 0)


def _places(s):
    """Where new row r of sequence i is stored: (page, place within the page, is there one)."""
    r = torch.arange(s["rows"], device=s["lengths"].device)
    n = _new(s)[:, None]
    p = s["lengths"].long()[:, None] - n + r
    there = (r < n) & (p >= 0)
    p = torch.where(there, p, 0)
    return s["table"].long().gather(1, p // PAGE), p % PAGE, there


def _plain_attend(s):
    q = s["q"]
    k, v = _gathered(s)
    S, R, H, d = q.shape
    G = k.shape[1]
    qg = q.float().view(S, R, G, H // G, d).permute(0, 2, 3, 1, 4).reshape(S, G, -1, d)
    x = torch.matmul(qg, k.transpose(-1, -2)).unflatten(2, (H // G, R)) / math.sqrt(d)
    x = x.masked_fill(torch.arange(k.shape[2], device=q.device) >= _limits(s)[:, None, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    # what a masked place holds is no number to rely on
    v = torch.where((torch.arange(k.shape[2], device=q.device) < s["lengths"][:, None])[:, None, :, None], v, 0.0)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (H // G, R)) / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log(total)).squeeze(-1)
    return out.permute(0, 3, 1, 2, 4).reshape(S, R, H, d).to(q.dtype), lse.permute(0, 3, 1, 2).reshape(S, R, H)


def _plain_store(s):
    page, slot, there = _places(s)
    d = s["dim"]
    G = s["k"].shape[2]
    tiles = s["pool"].view(-1, G, 2, s["pool"].shape[-1] // 2)
    a, b = d // 2, d // GROUP * 2
    at = torch.nonzero(there, as_tuple=True)
    pg, t, r = page[at], slot[at] // TILE, slot[at] % TILE
    heads = torch.arange(G, device=pg.device)
    for x, o in ((s["k"], 0), (s["v"], TILE * (a + b))):
        codes, scales = _quantise(x[at])
        for part, width, base in ((codes, a, o), (scales.view(torch.uint8), b, o + TILE * a)):
            place = base + r[:, None] * width + torch.arange(width, device=pg.device)
            tiles[pg[:, None, None], heads[None, :, None], t[:, None, None], place[:, None, :]] = part
    # the values of the stored rows, read back; zeros where a row has no place
    kc, ks, vc, vs = _parts(tiles[page[:, :, None], heads, (slot // TILE)[:, :, None]], d)
    pick = (slot % TILE)[:, :, None, None, None].expand(-1, -1, G, 1, -1)

    def of(x):
        return torch.gather(x, 3, pick.expand(-1, -1, -1, 1, x.shape[-1])).squeeze(3)

    keep = there[:, :, None, None]
    return tuple(torch.where(keep, _values(of(x), of(y)), 0.0).to(s["k"].dtype) for x, y in ((kc, ks), (vc, vs)))


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    if own:
        from moe_decode_megakernel_persistent_gb300 import kv4, pages
        if s["op"] == "copy":
            pages.copy(s["pool"], s["src"], s["dst"])
            return s["pool"]
        if s["op"] == "store":
            kv4.store(s["pool"], s["table"], s["lengths"], s["k"], s["v"], n_new=s["n_new"])
            return kv4.load(s["pool"], s["table"], s["lengths"], s["rows"], n_new=s["n_new"], dtype=s["k"].dtype)
        return kv4.attention(s["q"], s["pool"], s["table"], s["lengths"], n_new=s["n_new"], return_lse=True)
    if s["op"] == "copy":
        s["pool"][:, s["dst"]] = s["pool"][:, s["src"]]
        return s["pool"]
    return _plain_store(s) if s["op"] == "store" else _plain_attend(s)


def work(case):
    c = case
    if c["op"] == "copy":
        page = c["kv_heads"] * (_record(c["dim"]) if c["form"] == "4-bit" else 2 * PAGE * c["dim"] * 2)
        return {"bytes": 2 * c["layers"] * c["moves"] * page, "flops": 0}
    size = 2 if c["dtype"] == "bf16" else 4
    new, lengths, d = _n_new(c), _lengths(c), c["dim"]
    held = c["kv_heads"] * 2 * (d // 2 + d // GROUP * 2)        # bytes of one position
    if c["op"] == "store":
        n = sum(min(a, b) for a, b in zip(new, lengths))
        values = 2 * n * c["kv_heads"] * d
        # read, stored, loaded, and the values written
        return {"bytes": 2 * values * size + 2 * n * held, "flops": 4 * values}
    seen = sum(max(0, b - a + r + 1) for a, b in zip(new, lengths) for r in range(a))
    rows = c["seqs"] * c["rows"] * c["heads"]
    read = sum(b for a, b in zip(new, lengths) if a)
    return {"bytes": read * held + rows * (2 * d * size + 4), "flops": 4 * seen * c["heads"] * d}


# ---------------------------------------------------------------- in 64 bits

def _exact_rows(x):
    """What rows x [..., dim] read back as: the 4-bit rule, whose divisions are rounded to fp32 by its definition."""
    y = x.double().reshape(*x.shape[:-1], -1, GROUP)
    top = y.abs().max(-1, keepdim=True).values
    s = (top / 7).float().to(torch.bfloat16).double()
    m = torch.minimum(torch.round((y.abs() / s).float().double()), torch.tensor(7.0, dtype=torch.float64, device=x.device))
    return (torch.sign(y) * torch.where(s > 0, m, 0.0) * torch.where(s > 0, s, 0.0)).reshape(x.shape)


def _exact_cache(pool, pages, length, d):
    """K and V in 64 bits of one sequence, [kv heads, length, dim]."""
    raw = pool[pages].permute(1, 0, 2).reshape(pool.shape[1], -1, pool.shape[2] // 2)   # [G, tiles, bytes]
    half = raw.shape[-1] // 2
    got = []
    for part in (raw[..., :half], raw[..., half:]):
        code = part[..., :TILE * d // 2].reshape(raw.shape[0], -1, d // 2)
        scale = part[..., TILE * d // 2:].contiguous().view(torch.bfloat16).double().reshape(raw.shape[0], -1, d // GROUP)
        level = torch.tensor([0., 1, 2, 3, 4, 5, 6, 7, -0., -1, -2, -3, -4, -5, -6, -7], dtype=torch.float64, device=pool.device)
        x = torch.empty((*code.shape[:2], d), dtype=torch.float64, device=pool.device)
        x[..., 0::2] = level[(code % 16).long()]
        x[..., 1::2] = level[(code // 16).long()]
        got.append((x * scale.repeat_interleave(GROUP, -1))[:, :length])
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "copy":
        want = s["pool"].clone()
        for a, b in zip(s["src"], s["dst"]):
            want[:, b] = s["pool"][:, a]
        return want.double() if want.is_floating_point() else None
    new, lengths = _n_new(case), _lengths(case)
    if s["op"] == "store":
        out = []
        for x in (s["k"], s["v"]):
            y = _exact_rows(x)
            for i, (n, ln) in enumerate(zip(new, lengths)):
                y[i, n:] = 0
                y[i, :max(0, n - ln)] = 0
            out.append(y)
        return tuple(out)
    S, R, H, d = s["q"].shape
    out = torch.zeros((S, R, H, d), dtype=torch.float64, device="cuda")
    lse = torch.full((S, R, H), -math.inf, dtype=torch.float64, device="cuda")
    for i, (n, ln) in enumerate(zip(new, lengths)):
        k, v = _exact_cache(s["pool"], s["table"][i, :-(-ln // PAGE)].long(), ln, d)
        for r0 in range(max(0, n - ln), n, 128):
            r1 = min(n, r0 + 128)
            upto = ln - n + r1                                   # what the last of these rows sees
            for g in range(k.shape[0]):
                hs = slice(g * (H // k.shape[0]), (g + 1) * (H // k.shape[0]))
                x = torch.einsum("rhd,td->rht", s["q"][i, r0:r1, hs].double(), k[g, :upto]) / math.sqrt(d)
                sees = torch.arange(upto, device="cuda")[None, :] <= torch.arange(ln - n + r0, upto, device="cuda")[:, None]
                x = torch.where(sees[:, None, :], x, -math.inf)
                lse[i, r0:r1, hs] = torch.logsumexp(x, -1)
                out[i, r0:r1, hs] = torch.einsum("rht,td->rhd", torch.softmax(x, -1), v[g, :upto])
    return out, lse

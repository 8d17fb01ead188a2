"""The operators on the 16-bit paged cache restated in 64 bits, from their
description in include/mk.h (no code of the library), and how far fp32 may be off."""
import math

import torch

PAGE = 128


def table_for(lengths, spare=2, seed=0, width=None, device="cuda"):
    """Scattered pages for the lengths; unused entries are -1, which nothing may follow."""
    need = [-(-n // PAGE) for n in lengths]
    perm = torch.randperm(sum(need) + spare, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    t = torch.full((len(lengths), width or max(1, max(need, default=1))), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(need):
        t[i, :k] = perm[at:at + k]
        at += k
    return t.to(device), sum(need) + spare


def rows_of(pool, table, i, n):
    """K and V of sequence i's first n positions, float64 [n, heads, hd] each."""
    pages = pool[table[i, :-(-n // PAGE)].long()]
    return tuple(pages[:, j].permute(0, 2, 1, 3).flatten(0, 1)[:n].double() for j in (0, 1))


def put(pool, table, i, first, k, v):
    """Write k, v [n, heads, hd] into positions first .. of sequence i."""
    p = torch.arange(first, first + k.shape[0], device=pool.device)
    page = table[i].long()[p // PAGE]
    pool[page, 0, :, p % PAGE] = k.to(pool.dtype)
    pool[page, 1, :, p % PAGE] = v.to(pool.dtype)


def attend(q, k, v, first, scale, left_out=None):
    """Rows q [R, H, hd] at positions first .. first + R - 1 over k, v [n, G, hd] in float64.
    Returns out, lse, the weights w [R, H, n], A (the weights' sum of |v|) and D (the largest
    sum |scale q k| of a seen position), which the bounds need.  What a row does not see has
    weight 0, whatever its values."""
    R, H, hd = q.shape
    n, G, _ = k.shape
    q, kk, vv = q.double(), k.repeat_interleave(H // G, 1), v.repeat_interleave(H // G, 1)
    p = torch.arange(n, device=q.device)
    sees = p[None, :] <= (first + torch.arange(R, device=q.device))[:, None]
    if left_out is not None:
        sees = sees & ~left_out[None, :]
    sees = sees[:, None, :]
    s = (torch.einsum("rhd,nhd->rhn", q, kk) * scale).masked_fill(~sees, -math.inf)
    lse = torch.logsumexp(s, -1) if n else torch.full((R, H), -math.inf, dtype=torch.float64, device=q.device)
    w = torch.where(sees, torch.exp(s - lse.clamp(min=-1e300)[..., None]), 0.0)
    out, A = torch.zeros(R, H, hd, dtype=torch.float64, device=q.device), torch.zeros(R, H, hd, dtype=torch.float64, device=q.device)
    if torch.isfinite(vv).all():
        out, A = torch.einsum("rhn,nhd->rhd", w, vv), torch.einsum("rhn,nhd->rhd", w, vv.abs())
    else:
        for r in range(R):
            m = sees[r, 0]
            out[r] = torch.einsum("hn,nhd->hd", w[r][:, m], vv[m])
            A[r] = torch.einsum("hn,nhd->hd", w[r][:, m], vv[m].abs())
    D = (torch.einsum("rhd,nhd->rhn", q.abs(), kk.abs()) * abs(scale)).masked_fill(~sees, 0).amax(-1) if n else lse * 0
    return out, lse, w, A, D


def bounds(A, D, lse, n, hd, dtype):
    """How far out and lse may be off, by arithmetic.

    A score is a sum of hd products, exact in the products (an fp32 q of three bf16 parts is
    short of 2^-24 of each) and rounded at most 2 hd times in fp32 (2^-24 each, relative to
    the terms' sum D), scaled with a handful of roundings, and enters an exponential whose
    argument, of magnitude at most 2 D + |lse|, is rounded a few times and whose result is
    off by 2^-22: delta is the relative error of a weight.  Numerator and denominator sum n
    terms (n 2^-24 each at worst).  Weights enter the second product rounded to bf16 (half a
    step: 2^-8) for bf16 rows, in three parts (2^-24) for fp32 rows.  Returns the absolute
    bound of out before its own rounding, that rounding's relative bound, and lse's bound."""
    e = 2.0 ** -24
    delta = (2 * hd + 16) * e * D + 8 * e * (2 * D + 1) + 2.0 ** -21
    part = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    inner = A * (2 * delta + 2 * n * e + part + 8 * e)[..., None]
    return inner, torch.finfo(dtype).eps / 2, delta + n * e + 4 * e * (1 + lse.abs())


def mass_step(old, w, D, lse, n, hd, n_new, decay, gqa):
    """New masses of a sequence's n positions [G, n] and their bound: old [G, n] float64 and the
    weights w [R, H, n] of its real rows.  A weight e^(s - lse) has the relative error of a
    weight plus lse's absolute one; sums of R gqa terms in fp32 are off by 2^-24 for each."""
    e = 2.0 ** -24
    R, H, _ = w.shape
    delta = (2 * hd + 16) * e * D + 8 * e * (2 * D + 1) + 2.0 ** -21
    fine = torch.isfinite(lse)
    tau = 2 * delta + n * e + 12 * e * (1 + torch.where(fine, lse, 0.0).abs()) + (R * gqa + 4) * e
    keep = torch.arange(n, device=w.device) < n - n_new
    base = torch.where(keep, decay * old, 0.0)
    got = w.unflatten(1, (H // gqa, gqa)).sum((0, 2))
    off = (w * tau[..., None]).unflatten(1, (H // gqa, gqa)).sum((0, 2))
    # (a weight below 2^-126 is none in fp32's normal range: each may be lost whole)
    return base + got, off + 4 * e * base.abs() + e * got + R * gqa * 2.0 ** -126


def evict(mass, length, keep, recent):
    """kept [keep] (a list) of one sequence and head: the position that each slot then holds."""
    if length <= keep:
        return list(range(length)) + [-1] * (keep - length)
    others = [float(x) for x in mass[:length - recent]]
    rank = sorted(range(len(others)), key=lambda p: (-math.inf if math.isnan(others[p]) else 0, -others[p] if not math.isnan(others[p]) else 0, p))
    stays = set(rank[:keep - recent]) | set(range(length - recent, length))
    late = iter(sorted(p for p in stays if p >= keep))
    return [s if s in stays else next(late) for s in range(keep)]

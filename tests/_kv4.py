"""The 4-bit cache's format and its attention restated in 64 bits, from the
description in include/mk.h (no code of the library)."""
import math

import torch

PAGE, TILE, GROUP = 128, 64, 64


def record(hd):
    return 136 * hd


def quantise(x):
    """Codes (int64, sign in bit 3) [..., hd] and scales (bfloat16) [..., hd / 64]."""
    y = x.float().double().reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    top = y.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(y).all(-1, keepdim=True)
    # the definition divides in fp32; the fp64 quotient rounded to fp32 is that division
    s = torch.where(bad, torch.zeros_like(top), top / 7).float().to(torch.bfloat16)
    sd = s.double()
    m = torch.round((y.abs() / sd).float().double()).clamp(max=7)
    m = torch.where((sd > 0) & ~bad, m, torch.zeros_like(m)).long()
    code = m + 8 * ((y < 0) & (m > 0)).long()
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    return code.reshape(x.shape), s.squeeze(-1)


def values(code, scale):
    """What codes and scales stand for, float64."""
    v = (code & 7).double() * (1 - 2 * ((code >> 3) & 1).double())
    return (v.reshape(*v.shape[:-1], v.shape[-1] // GROUP, GROUP) * scale.double().unsqueeze(-1)).reshape(v.shape)


def put(pool, hd, page, slot, head, kv, code, scale):
    """Write one row's codes [hd] and scales into a CPU pool, byte by byte."""
    a, b = hd // 2, hd // GROUP * 2
    t, r = slot // TILE, slot % TILE
    base = t * TILE * 2 * (a + b) + kv * TILE * (a + b)
    rec = pool[page, head]
    rec[base + r * a: base + (r + 1) * a] = (code[0::2] + 16 * code[1::2]).to(torch.uint8)
    rec[base + TILE * a + r * b: base + TILE * a + (r + 1) * b] = scale.contiguous().view(torch.uint8)


def get(pool, hd, page, slot, head, kv):
    """(codes, scales) of one row of a CPU pool."""
    a, b = hd // 2, hd // GROUP * 2
    t, r = slot // TILE, slot % TILE
    base = t * TILE * 2 * (a + b) + kv * TILE * (a + b)
    raw = pool[page, head, base + r * a: base + (r + 1) * a].long()
    code = torch.stack((raw & 15, raw >> 4), -1).reshape(hd)
    return code, pool[page, head, base + TILE * a + r * b: base + TILE * a + (r + 1) * b].clone().view(torch.bfloat16)


def fill(pool, hd, pages, k, v):
    """Quantise k, v [positions, heads, hd] into the pages of a pool, all at once."""
    n, G, _ = k.shape
    pad = -n % PAGE
    parts = []
    for x in (k, v):
        x = torch.cat([x, x.new_zeros(pad, G, hd)])
        code, s = quantise(x)
        raw = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
        parts += [raw.reshape(-1, 2, TILE, G, hd // 2).permute(0, 3, 1, 2, 4).flatten(3),
                  s.contiguous().view(torch.uint8).reshape(-1, 2, TILE, G, hd // GROUP * 2).permute(0, 3, 1, 2, 4).flatten(3)]
    pool[pages] = torch.cat(parts, -1).flatten(2).to(pool.device)


def cache_values(pool, hd, pages, n):
    """K and V of n positions held in `pages`, float64 [n, heads, hd], on the pool's device."""
    a, b = TILE * hd // 2, TILE * hd // GROUP * 2
    raw = pool[pages].reshape(len(pages), pool.shape[1], 2, -1)        # [pages, heads, tiles, bytes]
    out = []
    for o in (0, a + b):
        code = raw[..., o:o + a].long().reshape(*raw.shape[:3], TILE, hd // 2)
        code = torch.stack((code & 15, code >> 4), -1).flatten(-2)
        s = raw[..., o + a:o + a + b].contiguous().view(torch.bfloat16).reshape(*raw.shape[:3], TILE, hd // GROUP)
        out.append(values(code, s).permute(0, 2, 3, 1, 4).reshape(-1, pool.shape[1], hd)[:n])
    return out


def attend(q, k, v, first, scale, left_out=None):
    """Rows q [R, H, hd] at positions first .. first + R - 1 over k, v [n, G, hd]
    in float64: (out, lse, A, D) with A the weights' sum of |v| and D a bound of
    the scores' magnitude sum |scale q k| for each row and head, which the
    error bounds need.  left_out: positions that no row sees."""
    R, H, hd = q.shape
    n, G, _ = k.shape
    q, kk, vv = q.double(), k.repeat_interleave(H // G, 1), v.repeat_interleave(H // G, 1)
    s = torch.einsum("rhd,nhd->rhn", q, kk) * scale
    p = torch.arange(n, device=q.device)
    sees = p[None, :] <= (first + torch.arange(R, device=q.device))[:, None]
    if left_out is not None:
        sees = sees & ~left_out[None, :]
    s = s.masked_fill(~sees[:, None, :], -math.inf)
    lse = torch.logsumexp(s, -1) if n else torch.full((R, H), -math.inf, dtype=torch.float64, device=q.device)
    w = torch.where(sees[:, None, :], torch.exp(s - lse.clamp(min=-1e300)[..., None]), 0.0)
    out = torch.einsum("rhn,nhd->rhd", w, vv)
    A = torch.einsum("rhn,nhd->rhd", w, vv.abs())
    D = (torch.einsum("rhd,nhd->rhn", q.abs(), kk.abs()) * abs(scale)).masked_fill(~sees[:, None, :], 0).amax(-1) if n else lse * 0
    return out, lse, A, D


def bounds(A, D, lse, n, hd, dtype, top):
    """How far out and lse may be off, by arithmetic.

    A score is a sum of hd products, exact in the products and rounded at most
    2 hd times in fp32 (2^-24 each, relative to the terms' sum D), scaled with a
    handful of roundings, and then enters an exponential whose argument, of
    magnitude at most 2 D + |lse|, is rounded a few times and whose result is off
    by 2^-22: delta below is the relative error of a weight.  Numerator and
    denominator sum n terms (n 2^-24 each at worst).  For bf16 rows the weights
    enter the second product rounded to fp16 (half a step: 2^-11), for fp32 rows
    in two fp16 parts (2^-22).  fp16 ends at 2^-25 in absolute terms, where the
    weights are normalised so that the largest possible term is 2^6 to 2^14: a
    term is off by 2^-28 of the largest scale's (2^-27 covers it), fp32 rows' low
    parts likewise.  top is the largest |value| / 7, at least the largest scale."""
    e = 2.0 ** -24
    delta = (2 * hd + 16) * e * D + 8 * e * (2 * D + 1) + 2.0 ** -21
    part = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22
    inner = A * (2 * delta + 2 * n * e + part + 8 * e)[..., None] + n * 2.0 ** -27 * top
    # the result's own rounding: half a step of its type
    return inner, torch.finfo(dtype).eps / 2, delta + n * e + 4 * e * (1 + lse.abs())

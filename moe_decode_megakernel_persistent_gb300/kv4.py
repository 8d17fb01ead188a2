"""A paged K/V cache held in 4 bits: store, load and attention over torch
tensors (mk_kv4_store, mk_kv4_load and mk_kv4_attention of include/mk.h, which
describes the format; argument checks and marshalling only).

A pool of one layer is a uint8 CUDA tensor [n_pages, n_kv_heads, record]
(`new_pool`; one layer of a pool of several is `pool[l]`).  table is int32
[n_seqs, max_pages], lengths int32 [n_seqs], n_new int32 [n_seqs] or None, all
on the pool's device.  Sequence i holds lengths[i] positions, position p in slot
p % 128 of page table[i, p // 128]; its n_new[i] new rows (all rows of the call
without n_new) are the last of them, and rows past n_new[i] are padding.

Calls run on the current stream of the pool's device and return before the work
is done.  They can be captured into a CUDA graph, which reads table, lengths and
n_new anew at every replay.  A length, n_new or page outside its range is
reported in `status` (a zeroed int32 CUDA tensor of one element) as
MK_ERR_DEVICE_INDEX and never read or written past.
"""
from __future__ import annotations

import math

import torch

from . import _lib as L

PAGE_TOKENS = 128
_DT = {torch.bfloat16: L.MK_BF16, torch.float32: L.MK_F32}


def new_pool(n_pages: int, n_kv_heads: int, head_dim: int, n_layers: int | None = None, device="cuda") -> torch.Tensor:
    """A pool of zeros: [n_pages, n_kv_heads, record], or with n_layers
    [n_layers, n_pages, n_kv_heads, record]."""
    nbytes = L.mk_kv4_page_bytes(n_kv_heads, head_dim)
    if nbytes == 0 or n_pages < 1:
        raise ValueError("n_pages and n_kv_heads must be >= 1 and head_dim 64 or 128")
    lead = (n_pages,) if n_layers is None else (n_layers, n_pages)
    return torch.zeros((*lead, n_kv_heads, nbytes // n_kv_heads), dtype=torch.uint8, device=device)


def _int32(t, shape, dev, what):
    if t.dtype != torch.int32 or t.device != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {tuple(shape)} on {dev}")
    return t.data_ptr()


def _cache(pool, table, lengths, n_new, status, rows, head_dim) -> L.mk_kv4_cache:
    dev = pool.device
    if not pool.is_cuda or pool.dtype != torch.uint8 or pool.dim() != 3 or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous uint8 CUDA tensor [n_pages, n_kv_heads, record]")
    if pool.shape[2] != head_dim * 136:
        raise ValueError(f"a record of {pool.shape[2]} bytes does not hold heads of {head_dim}")
    if table.dim() != 2:
        raise ValueError("table must be int32 [n_seqs, max_pages]")
    n, width = table.shape
    return L.mk_kv4_cache(pool.data_ptr(), _int32(table, (n, width), dev, "table"), _int32(lengths, (n,), dev, "lengths"),
                          None if n_new is None else _int32(n_new, (n,), dev, "n_new"),
                          None if status is None else _int32(status, (1,), dev, "status"),
                          pool.shape[0], pool.shape[1], head_dim, n, width, rows)


def _rows(x, pool, n, what) -> L.mk_kv4_rows:
    if x.dim() != 4 or x.shape[0] != n or x.device != pool.device or x.dtype not in _DT:
        raise ValueError(f"{what} must be bfloat16 or float32 [n_seqs = {n}, rows, heads, head_dim] on {pool.device}")
    s = x.stride()
    if s[3] != 1 and x.shape[3] != 1:
        raise ValueError(f"{what}: head_dim must be contiguous")
    return L.mk_kv4_rows(x.data_ptr(), *(s[i] if x.shape[i] > 1 else 0 for i in range(3)))


def _on(dev):
    """The device's current stream; the device made current around the call."""
    return torch.cuda.device(dev), torch.cuda.current_stream(dev).cuda_stream


def store(pool, table, lengths, k, v, n_new=None, status=None):
    """Store the new rows' K and V, [n_seqs, rows, n_kv_heads, head_dim] each
    (any strides that are multiples of 16 bytes, head_dim contiguous), in their
    places.  Two sequences must not store in the same place."""
    kr, vr = _rows(k, pool, table.shape[0], "k"), _rows(v, pool, table.shape[0], "v")
    if k.shape != v.shape or k.dtype != v.dtype or k.shape[2] != pool.shape[1]:
        raise ValueError("k and v must have one shape and dtype, and the pool's kv heads")
    c = _cache(pool, table, lengths, n_new, status, k.shape[1], k.shape[3])
    guard, st = _on(pool.device)
    with guard:
        L.mk_kv4_store(c, kr, vr, _DT[k.dtype], st)


def load(pool, table, lengths, rows: int, n_new=None, dtype=torch.bfloat16, status=None):
    """(k, v) of the new rows' places, [n_seqs, rows, n_kv_heads, head_dim];
    zeros in padding rows.  With rows = the largest length and n_new = lengths
    it reads whole sequences."""
    if dtype not in _DT:
        raise ValueError("dtype must be bfloat16 or float32")
    if rows < 0:
        raise ValueError("rows must be >= 0")
    hd = pool.shape[-1] // 136
    c = _cache(pool, table, lengths, n_new, status, rows, hd)
    k, v = (torch.empty((c.n_seqs, rows, c.n_kv_heads, hd), dtype=dtype, device=pool.device) for _ in range(2))
    guard, st = _on(pool.device)
    with guard:
        L.mk_kv4_load(c, _rows(k, pool, c.n_seqs, "k"), _rows(v, pool, c.n_seqs, "v"), _DT[dtype], st)
    return k, v


def attention(q, pool, table, lengths, n_new=None, scale=None, out=None, return_lse=False, status=None):
    """Causal attention of the new rows q [n_seqs, rows, n_heads, head_dim] over
    the cache, which holds their own K and V already.  scale defaults to
    1 / sqrt(head_dim).  Returns out in q's dtype (`out` if given), with
    return_lse also the log-sum-exp of the scores, float32 [n_seqs, rows,
    n_heads].  Rows that see nothing are zeros, with a log-sum-exp of -inf."""
    n = table.shape[0]
    qr = _rows(q, pool, n, "q")
    c = _cache(pool, table, lengths, n_new, status, q.shape[1], q.shape[3])
    heads = q.shape[2]
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != q.device or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape, dtype and device")
    lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device) if return_lse else None
    dt = _DT[q.dtype]
    nws = L.mk_kv4_attention_bytes(c, heads, dt)
    # taken anew for each call from the stream's allocator, so that calls on two
    # streams, or two captured graphs, never share one
    ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
    guard, st = _on(pool.device)
    with guard:
        L.mk_kv4_attention(c, heads, qr, dt, 1.0 / math.sqrt(q.shape[3]) if scale is None else scale,
                           _rows(out, pool, n, "out"), None if lse is None else lse.data_ptr(),
                           None if ws is None else ws.data_ptr(), nws, st)
    return (out, lse) if return_lse else out

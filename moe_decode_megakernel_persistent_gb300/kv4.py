"""A paged K/V cache held in 4 bits: store, load and attention over torch
tensors (mk_kv4_store, mk_kv4_load and mk_kv4_attention of include/mk.h, which
describes the format; the checks of the tensors and the calls are csrc/mk_torch.cpp).

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

They have no gradient: a q, k, v or out that requires one is refused (call them
under torch.no_grad(), or detach the tensor).
"""
from __future__ import annotations

import torch

from . import _lib as L

PAGE_TOKENS = 128
_BF16 = {torch.bfloat16: True, torch.float32: False}


def new_pool(n_pages: int, n_kv_heads: int, head_dim: int, n_layers: int | None = None, device="cuda") -> torch.Tensor:
    """A pool of zeros: [n_pages, n_kv_heads, record], or with n_layers
    [n_layers, n_pages, n_kv_heads, record]."""
    nbytes = L.mk_kv4_page_bytes(n_kv_heads, head_dim)
    if nbytes == 0 or n_pages < 1:
        raise ValueError("n_pages and n_kv_heads must be >= 1 and head_dim 64 or 128")
    lead = (n_pages,) if n_layers is None else (n_layers, n_pages)
    return torch.zeros((*lead, n_kv_heads, nbytes // n_kv_heads), dtype=torch.uint8, device=device)


def store(pool, table, lengths, k, v, n_new=None, status=None):
    """Store the new rows' K and V, [n_seqs, rows, n_kv_heads, head_dim] each
    (any strides that are multiples of 16 bytes, head_dim contiguous), in their
    places.  Two sequences must not store in the same place."""
    L.torch_module().store(pool, table, lengths, k, v, n_new, status)


def load(pool, table, lengths, rows: int, n_new=None, dtype=torch.bfloat16, status=None):
    """(k, v) of the new rows' places, [n_seqs, rows, n_kv_heads, head_dim];
    zeros in padding rows.  With rows = the largest length and n_new = lengths
    it reads whole sequences."""
    bf16 = _BF16.get(dtype)
    if bf16 is None:
        raise ValueError("dtype must be bfloat16 or float32")
    return L.torch_module().load(pool, table, lengths, rows, n_new, bf16, status)


def attention(q, pool, table, lengths, n_new=None, scale=None, out=None, return_lse=False, status=None):
    """Causal attention of the new rows q [n_seqs, rows, n_heads, head_dim] over
    the cache, which holds their own K and V already.  scale defaults to
    1 / sqrt(head_dim).  Returns out in q's dtype (`out` if given: contiguous, and
    of memory that neither q nor the pool has), with
    return_lse also the log-sum-exp of the scores, float32 [n_seqs, rows,
    n_heads].  Rows that see nothing are zeros, with a log-sum-exp of -inf.  The
    work is split by the table's width: short sequences are faster in a table
    that is not far wider than they need."""
    return L.torch_module().attention(q, pool, table, lengths, n_new, scale, out, bool(return_lse), status)

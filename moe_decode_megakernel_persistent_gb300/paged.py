"""Operators on a paged 16-bit K/V cache held by torch tensors: store, attention of
single rows and chunks, the weights that cached positions receive, and the
eviction of those that received least (mk_paged_store, mk_paged_attention and
mk_paged_evict of include/mk.h; the checks of the tensors and the calls are
csrc/mk_torch.cpp).

A pool of one layer is a bfloat16 CUDA tensor [n_pages, 2, n_kv_heads, 128,
head_dim] (`new_pool`; one layer of a pool of several is `pool[l]`), the layout of
the engine's own cache (which stays inside the engine).  table is int32 [n_seqs, max_pages], lengths int32
[n_seqs], n_new int32 [n_seqs] or None, all on the pool's device.  Sequence i
holds lengths[i] positions, position p in slot p % 128 of page table[i, p // 128];
its n_new[i] new rows (all rows of the call without n_new) are the last of them,
and rows past n_new[i] are padding.

Calls run on the current stream of the pool's device and return before the work
is done.  They can be captured into a CUDA graph, which reads table, lengths and
n_new anew at every replay.  A length, n_new or page outside its range is
reported in `status` (a zeroed int32 CUDA tensor of one element) as
MK_ERR_DEVICE_INDEX and never read or written past.

They have no gradient: a tensor that requires one is refused (call them under
torch.no_grad(), or detach the tensor).

A cache on a budget, a token at a time (the positions of the rotary embedding are
the caller's, and go on counting):

    mass = paged.new_mass(table, n_kv_heads)
    paged.store(pool, table, lengths, k, v)
    out = paged.attention(q, pool, table, lengths, mass=mass)
    paged.evict(pool, table, lengths, mass, keep=4096, recent=256, new_lengths=lengths, new_mass=mass)
"""
from __future__ import annotations

import torch

from . import _lib as L

PAGE_TOKENS = 128


def new_pool(n_pages: int, n_kv_heads: int, head_dim: int, n_layers: int | None = None, device="cuda") -> torch.Tensor:
    """A pool of zeros: [n_pages, 2, n_kv_heads, 128, head_dim], or with n_layers
    [n_layers, n_pages, 2, n_kv_heads, 128, head_dim]."""
    if n_pages < 1 or n_kv_heads < 1 or head_dim not in (64, 128):
        raise ValueError("n_pages and n_kv_heads must be >= 1 and head_dim 64 or 128")
    lead = (n_pages,) if n_layers is None else (n_layers, n_pages)
    return torch.zeros((*lead, 2, n_kv_heads, PAGE_TOKENS, head_dim), dtype=torch.bfloat16, device=device)


def new_mass(table: torch.Tensor, n_kv_heads: int) -> torch.Tensor:
    """Masses of zeros for the sequences and pages of a table: float32 [n_seqs,
    n_kv_heads, 128 * max_pages]."""
    return torch.zeros((table.shape[0], n_kv_heads, PAGE_TOKENS * table.shape[1]), device=table.device)


def store(pool, table, lengths, k, v, n_new=None, status=None):
    """Store the new rows' K and V, [n_seqs, rows, n_kv_heads, head_dim] of
    bfloat16 or float32 (any strides that are multiples of 16 bytes, head_dim
    contiguous), in their places, rounded to bfloat16.  Two sequences must not
    store in the same place."""
    L.torch_module().paged_store(pool, table, lengths, k, v, n_new, status)


def attention(q, pool, table, lengths, n_new=None, scale=None, out=None, return_lse=False, mass=None, decay=1.0,
              status=None):
    """Causal attention of the new rows q [n_seqs, rows, n_heads, head_dim]
    (bfloat16 or float32) over the cache, which holds their own K and V already.
    scale defaults to 1 / sqrt(head_dim).  Returns out in q's dtype (`out` if
    given: contiguous, and of memory that neither q, the pool nor mass has), with
    return_lse also the log-sum-exp of the scores, float32 [n_seqs, rows,
    n_heads].  Rows that see nothing are zeros, with a log-sum-exp of -inf.

    mass (float32 [n_seqs, n_kv_heads, 128 * max_pages], positions contiguous):
    what each position has received.  For every sequence with a new row the
    masses of its earlier positions are multiplied by decay, those of its new
    positions start from 0, and each gets the sum of the weights that the rows and
    the query heads of its kv head give it.  Calls of few rows (at most 32 rows x
    query heads of a kv head) keep their scores meanwhile: 4 bytes for each of these,
    rounded up to a multiple of 4, and each kv head and position of the tables."""
    return L.torch_module().paged_attention(q, pool, table, lengths, n_new, scale, out, bool(return_lse), mass, decay, status)


def evict(pool, table, lengths, mass, keep: int, recent: int = 0, new_lengths=None, new_mass=None, status=None):
    """Leave at most `keep` positions of each (sequence, kv head): of a longer
    sequence the last `recent` ones and the heaviest others, ties to the lower
    position.  Kept positions below `keep` stay in their slots; the others' K and V
    move, in order, into the free slots below `keep`.  The pages of the first `keep`
    positions are written: no other sequence may share them, nor may the table name
    them twice.  Tables of at most 6144 pages.

    Returns (kept, new_lengths, new_mass): int32 [n_seqs, n_kv_heads, keep], the
    position that each slot now holds (-1 behind the end of a shorter sequence);
    int32 [n_seqs], min(length, keep); and the masses moved along, 0 behind the new
    length.  new_lengths and new_mass may be given, also as lengths and mass
    themselves (masses behind the new length then stay)."""
    return L.torch_module().paged_evict(pool, table, lengths, mass, keep, recent, new_lengths, new_mass, status)

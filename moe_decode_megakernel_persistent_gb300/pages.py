"""Page moves in a paged pool held by a torch tensor (mk_page_copy of
include/mk.h; argument checks and marshalling only)."""
from __future__ import annotations

import torch

from . import _lib as L


def copy(pool: torch.Tensor, src, dst):
    """Copy page src[i] to page dst[i] in every layer of pool, a contiguous CUDA
    tensor [n_layers, n_pages, ...] of any dtype whose pages are multiples of
    16 bytes.  src, dst: host lists of the same length; destinations are
    distinct and none is a source (the moves run at once).  Runs on the current
    stream of the pool's device; a captured graph repeats these very moves."""
    if not pool.is_cuda or pool.dim() < 3 or not pool.is_contiguous():
        raise ValueError("pool must be a contiguous CUDA tensor [n_layers, n_pages, ...]")
    if len(src) != len(dst):
        raise ValueError("src and dst must have the same length")
    if pool.shape[0] == 0 or pool.shape[1] == 0:
        raise ValueError("pool has no page")
    with torch.cuda.device(pool.device):
        L.mk_page_copy(pool.data_ptr(), pool.shape[0], pool.shape[1], pool[0, 0].numel() * pool.element_size(), src, dst,
                       torch.cuda.current_stream(pool.device).cuda_stream)

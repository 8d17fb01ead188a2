"""Page moves in a paged pool held by a torch tensor (mk_page_copy of
include/mk.h; the checks of the tensor and the call are csrc/mk_torch.cpp)."""
from __future__ import annotations

import torch

from . import _lib as L


def copy(pool: torch.Tensor, src, dst):
    """Copy page src[i] to page dst[i] in every layer of pool, a contiguous CUDA
    tensor [n_layers, n_pages, ...] of any dtype whose pages are multiples of
    16 bytes.  src, dst: host lists of the same length; destinations are
    distinct and none is a source (the moves run at once).  Runs on the current
    stream of the pool's device; a captured graph repeats these very moves.  A pool
    that requires a gradient is refused."""
    L.torch_module().page_copy(pool, src, dst)

"""The tensor calls of kv4 and pages have no gradient: what requires one is refused before anything
else about the call is looked at, and nothing else is."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from moe_decode_megakernel_persistent_gb300 import _build, kv4, pages


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()


def calls():
    """Calls whose first refusal, of CPU tensors, is the pool's device."""
    x = lambda: torch.zeros((1, 1, 2, 64))
    pool, i = torch.zeros((1, 2, 136 * 64), dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)
    table = i.view(1, 1)
    yield "q", x(), lambda t: kv4.attention(t, pool, table, i)
    yield "out", x(), lambda t: kv4.attention(x(), pool, table, i, out=t)
    yield "k", x(), lambda t: kv4.store(pool, table, i, t, x())
    yield "v", x(), lambda t: kv4.store(pool, table, i, x(), t)
    yield "pool", torch.zeros((1, 4, 64)), lambda t: pages.copy(t, [0], [1])


@pytest.mark.parametrize("at", range(5))
def test_what_requires_a_gradient_is_refused(at):
    name, t, call = list(calls())[at]
    other = "pool must be a contiguous"
    with pytest.raises(ValueError, match=other):
        call(t)
    leaf = t.clone().requires_grad_()
    for g in (leaf, leaf * 2):
        with pytest.raises(ValueError, match=f"{name} requires a gradient"):
            call(g)
        with pytest.raises(ValueError, match=other):
            call(g.detach())
        with torch.no_grad(), pytest.raises(ValueError, match=other):
            call(g)
    with fwd.dual_level():
        with pytest.raises(ValueError, match=f"{name} requires a gradient"):
            call(fwd.make_dual(t, torch.ones_like(t)))

"""A layer's buffers, planned for more tokens than a call has."""
from __future__ import annotations

import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import expert_layer  # noqa: E402


def test_fewer_tokens_than_planned():
    """The same launches as with a plan of their own, so the same bits, whatever a call with
    more tokens left in the buffers."""
    layer = expert_layer.random_layer(12, 256, 128, 3, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dout = (torch.randn(70, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    b = layer.plan(70)
    layer.forward(x, b)
    for n in (33, 1, 70, 0):
        own = layer.plan(n)
        want = layer.forward(x[:n], own).clone()
        got = layer.forward(x[:n], b)
        assert got.shape == (n, 256) and torch.equal(got, want)
        dx, dl = layer.backward(dout[:n], b)
        dx_want, dl_want = layer.backward(dout[:n], own)
        assert torch.equal(dx, dx_want) and torch.equal(dl, dl_want)


def test_more_tokens_than_planned_are_refused():
    layer = expert_layer.random_layer(4, 256, 128, 2, seed=5)
    with pytest.raises(ValueError):
        layer.forward(torch.zeros(9, 256, dtype=torch.bfloat16, device="cuda"), layer.plan(8))

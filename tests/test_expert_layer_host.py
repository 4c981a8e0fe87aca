"""What examples/expert_layer.py checks before it launches anything (CPU; the library's calls are
replaced by ones that look at their arguments)."""
from __future__ import annotations

import inspect
import os
import sys
import types

import pytest

import block_scaled_precision_bf16tofp4row_amd as mx

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import expert_layer  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    """The names of the calls so far, none of which may have offsets past its first operand's
    rows: the kernels would read behind it."""
    made = []

    def stand_in(name):
        fn = getattr(mx, name)
        if not name.startswith("mxfp4_") or name.endswith("_workspace"):
            return fn
        sig = inspect.signature(fn)

        def call(*args, **kw):
            a = sig.bind(*args, **kw).arguments
            rows = next(iter(a.values())).shape[0]
            if "offs" in a and name != "mxfp4_expert_map":
                assert int(a["offs"][-1]) <= rows, (name, a["offs"].tolist(), rows)
            made.append(name)

        return call

    stub = types.SimpleNamespace(**{n: stand_in(n) for n in dir(mx) if n.startswith(("mxfp4_", "alloc_"))})
    real = stub.alloc_fp8_rows_f32_outputs
    stub.alloc_fp8_rows_f32_outputs = lambda rows, k, device="cpu": real(rows, k, "cpu")
    monkeypatch.setattr(expert_layer, "mx", stub)
    return made


def dense(H=64, I=128):
    return expert_layer.FeedForward(torch.randn(2 * I, H), torch.randn(H, I), torch.randn(2 * I), torch.randn(H))


def rows(n, H=64):
    return torch.randn(n, H).bfloat16()


def test_dense_block_refuses_other_rows_than_planned(calls):
    block = dense()
    b = block.plan(20, device="cpu")
    for n in (0, 1, 19, 21):
        with pytest.raises(ValueError, match="planned for"):
            block.forward(rows(n), b)
    block.forward(rows(20), b, residual=rows(20))
    for n in (0, 1, 19, 21):
        with pytest.raises(ValueError, match="planned for"):
            block.backward(rows(n), b)
    with pytest.raises(ValueError, match="planned for"):
        block.backward(rows(20, 48), b)
    assert len(calls) == 3
    block.backward(rows(20), b)
    assert len(calls) == 7

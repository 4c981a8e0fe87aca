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
            if name == "mxfp4_expert_map":        # every choice has a row, all of the first expert
                a["offs"].fill_(a["pos"].numel())[0] = 0
                a["pos"].copy_(torch.arange(a["pos"].numel()).view_as(a["pos"]))
            elif "offs" in a:
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


def layer(fused):
    return expert_layer.random_layer(4, 64, 128, 2, seed=1, device="cpu", fused=fused)


def test_gradients_of_rows_that_were_not_kept_are_refused(calls):
    """Without keep a fused layer writes no h: the plan's is an earlier call's, or none."""
    m = layer(True)
    b = m.plan(9, device="cpu")
    with pytest.raises(ValueError, match="forward"):
        m.backward(rows(9), b)
    m.forward(rows(9), b)
    m.forward(rows(9), b, keep=False)
    with pytest.raises(ValueError, match="forward"):
        m.backward(rows(9), b)
    with pytest.raises(ValueError, match="backward"):
        m.weight_gradients(rows(9), b)
    assert "mxfp4_combine_rows_backward" not in calls
    m.forward(rows(9), b)
    m.backward(rows(9), b)
    assert "mxfp4_fp8_gated_gemm_backward" in calls


@pytest.mark.parametrize("fused", [True, False])
def test_gradients_of_other_tokens_are_refused(calls, fused):
    """The map in the plan is the last forward call's."""
    m = layer(fused)
    b = m.plan(9, device="cpu")
    m.forward(rows(7), b)
    for n in (0, 6, 8, 9):
        with pytest.raises(ValueError, match="forward"):
            m.backward(rows(n), b)
    m.backward(rows(7), b)
    if not fused:
        with pytest.raises(ValueError, match="backward"):
            m.weight_gradients(rows(7), b)
        return
    for n in (6, 8):
        with pytest.raises(ValueError, match="backward"):
            m.weight_gradients(rows(n), b)
    m.forward(rows(7), b)
    with pytest.raises(ValueError, match="backward"):
        m.weight_gradients(rows(7), b)


def test_dense_block_gradients_follow_a_forward_call(calls):
    block = dense()
    b = block.plan(5, device="cpu")
    with pytest.raises(ValueError, match="forward"):
        block.backward(rows(5), b)
    block.forward(rows(5), b)
    block.backward(rows(5), b)

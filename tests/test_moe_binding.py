"""What the binding keeps between calls (CPU): a size by its numbers alone."""

import pytest

import block_scaled_precision_bf16tofp4row_amd as mx

torch = pytest.importorskip("torch")


def test_workspace_size_of_a_tensor_that_changes():
    """The sizes may come as anything that has an int: what is kept goes by the number, not by
    the object that held it once."""
    T = torch.tensor(300)
    few = mx.mxfp4_expert_map_workspace(T, 8, 64)
    T.fill_(9000)
    many = mx.mxfp4_expert_map_workspace(T, 8, 64)
    assert few == mx.mxfp4_expert_map_workspace(300, 8, 64)
    assert many == mx.mxfp4_expert_map_workspace(9000, 8, 64) > few
    assert mx.mxfp4_expert_map_workspace(T=9000, k=8, G=64) == many

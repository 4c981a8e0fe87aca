"""The gated call's weight scales (CPU): blocks of a part, not of the joined features."""
from __future__ import annotations

import pytest

import block_scaled_precision_bf16tofp4row_amd as mx

torch = pytest.importorskip("torch")


def call(I, scales, joined=True, G=2, M=4, K=256):
    w = torch.zeros((G, 2 * I, K) if joined else (G, 2, I, K), dtype=torch.uint8)
    mx.mxfp4_fp8_gated_gemm(torch.zeros((M, K), dtype=torch.uint8), torch.zeros(M, 2), w, scales,
                            torch.zeros(G + 1, dtype=torch.int32), out=torch.zeros((M, I), dtype=torch.bfloat16))


@pytest.mark.parametrize("joined", [True, False])
@pytest.mark.parametrize("I", [72, 104, 120, 200, 248])
def test_scales_of_joined_features_are_refused(I, joined):
    """Blocks over the 2 I joined features are as many as those of both parts where the parts end
    in the second half of a block, but other rows'."""
    rows = -(-2 * I // 128)
    assert rows == 2 * -(-I // 128)
    for shape in ((2, rows, 2), (2 * rows, 2), (4 * rows,), (2, 1, rows, 2)):
        with pytest.raises(ValueError, match="w_scales has shape"):
            call(I, torch.zeros(shape), joined)
    with pytest.raises(ValueError, match="must be a GPU tensor"):         # past the check
        call(I, torch.zeros(2, 2, rows // 2, 2), joined)


@pytest.mark.parametrize("I", [64, 128, 136, 192, 256, 680])
def test_scales_that_cannot_be_mistaken(I):
    """Elsewhere the joined features have the parts' blocks, or fewer than both parts."""
    nb = -(-I // 128)
    for shape in ((2, 2, nb, 2), (2, 2 * nb, 2)):
        with pytest.raises(ValueError, match="must be a GPU tensor"):
            call(I, torch.zeros(shape))
    if I % 128:
        assert -(-2 * I // 128) < 2 * nb
        with pytest.raises(ValueError, match="w_scales holds"):
            call(I, torch.zeros(2, -(-2 * I // 128), 2))

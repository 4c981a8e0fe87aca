"""The combine's gradients where a wave's lanes exchange most through LDS: up to 64 choices, many
of them without a row, with one, four and sixteen waves per token; and the map's counters when
all 64 lanes of a step want the same one.

dy: one FP32 product, one rounding, so bit for bit.  dweights: K 2^-24 of the sum of magnitudes.
"""
from __future__ import annotations

import numpy as np
import pytest

import moe_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402


@pytest.mark.parametrize("T,K", [(9, 8), (50, 512), (7, 1032), (300, 520), (5, 2056), (3, 7168)])
@pytest.mark.parametrize("k,share", [(1, 1.0), (8, 1.0), (9, 0.5), (64, 1.0), (64, 0.3), (33, 0.0)])
def test_gradients(T, K, k, share):
    g = torch.Generator().manual_seed(T * K + k)
    slots = torch.randperm(T * k, generator=g).to(torch.int32).view(T, k)
    pos = torch.where(torch.rand(T, k, generator=g) < share, slots, -1)
    y, dout = (torch.randn(n, K, generator=g).bfloat16() for n in (T * k, T))
    w = torch.randn(T, k, generator=g)
    dy = torch.full((T * k, K), -3.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T, k), torch.nan, device="cuda")
    mx.mxfp4_combine_rows_backward(dout.cuda(), y.cuda(), pos.cuda(), w.cuda(), dy, dw)
    live = pos >= 0
    want = torch.full((T * k, K), -3.0).bfloat16()
    at = pos[live].long()
    want[at] = (w[live][:, None] * dout.float().repeat_interleave(k, 0).view(T, k, K)[live]).bfloat16()
    assert torch.equal(dy.cpu(), want)
    rows = y.double()[pos.clamp_min(0).long()]
    exact = (rows * dout.double()[:, None]).sum(2)
    mag = (rows * dout.double()[:, None]).abs().sum(2)
    got = dw.cpu().double()
    assert (got[~live] == 0).all()
    assert ((got - exact).abs() <= K * 2.0 ** -24 * mag)[live].all()


@pytest.mark.parametrize("T,k", [(300, 4), (5000, 3)])                        # one launch, two
def test_map_of_repeated_experts(T, k):
    """Runs of one expert longer than a step, then steps that alternate between two."""
    slot = np.arange(T * k)
    ids = np.where(slot // 200 % 2 == 0, 5, slot % 2).astype(np.int32).reshape(T, k)
    offs, pos, ws = mx.alloc_expert_map_outputs(T, k, 8)
    src = torch.empty(T * k, dtype=torch.int32, device="cuda")
    mx.mxfp4_expert_map(torch.from_numpy(ids).cuda(), offs, pos, ws, src=src)
    roffs, rpos, rsrc = ref.expert_map(ids, 0, 8, T * k)
    assert np.array_equal(offs.cpu().numpy(), roffs)
    assert np.array_equal(pos.cpu().numpy(), rpos) and np.array_equal(src.cpu().numpy(), rsrc)

"""Activations and their derivatives on the GPU, where the feed-forward calls give their FP32
values: a derivative as the bias gradient of one row of ones, an activation as the scale of an
E4M3 block whose other values are zero."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import act_bounds as ab  # noqa: E402
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402
import ffn_ref as fr  # noqa: E402

NAN, INF = float("nan"), float("inf")
#: the derivatives at NaN, +inf and -inf (where infinity times zero is in the formula: NaN)
SPECIAL = {"silu": (NAN, NAN, NAN), "gelu": (NAN, NAN, NAN), "gelu_tanh": (NAN, 1, 0), "relu": (NAN, 1, 0),
           "none": (1, 1, 1)}
#: and the activations
SPECIAL_VALUE = {"silu": (NAN, INF, NAN), "gelu": (NAN, INF, NAN), "gelu_tanh": (NAN, INF, NAN), "relu": (NAN, INF, 0),
                 "none": (NAN, INF, -INF)}


def slopes(x, act):
    """act' of BF16 numbers in FP32: one row per expert."""
    rows, n = x.shape
    x = x.cuda()
    offs = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    db = torch.full((rows, n), -3.0, device="cuda")
    ws = torch.empty(max(16, mx.mxfp4_act_rows_backward_workspace(rows, rows, n)), dtype=torch.uint8, device="cuda")
    mx.mxfp4_act_rows_backward(torch.ones_like(x), x, offs, dbias=db, workspace=ws, act=act)
    return db.cpu().numpy()


@pytest.mark.parametrize("act", SPECIAL)
def test_special_arguments(act):
    """NaN stays NaN, also as a derivative and also under ReLU; infinities as documented."""
    special = torch.tensor([NAN, INF, -INF] + [0.5] * 5, dtype=torch.bfloat16)[None].repeat(2, 1)
    want = np.array(SPECIAL[act], np.float32)
    assert np.array_equal(slopes(special, act)[:, :3], want[None].repeat(2, 0), equal_nan=True)
    # the gated product's gradient with d = 1 and up = 1: dh = [act'(g), act(g)], out = act(g)
    M, I, K = 2, 8, 16
    a, w = torch.zeros((M, K), dtype=torch.uint8, device="cuda"), torch.zeros((1, I, K), dtype=torch.uint8, device="cuda")
    a[:, 0], w[:, :, 0] = 0x38, 0x38              # E4M3 of 1
    sa, sw = torch.ones((M, 1), device="cuda"), torch.ones((1, 1, 1), device="cuda")
    h = torch.cat([special, torch.ones_like(special)], 1).cuda()
    dh, out = torch.full_like(h, -3), torch.full((M, I), -3.0, dtype=torch.bfloat16, device="cuda")
    offs = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    mx.mxfp4_fp8_gated_gemm_backward(a, sa, w, sw, h, offs, dh=dh, out=out, act=act)
    value = np.array(SPECIAL_VALUE[act], np.float32)[None].repeat(2, 0)
    got = dh.float().cpu().numpy()
    assert np.array_equal(got[:, :3], want[None].repeat(2, 0), equal_nan=True)
    assert np.array_equal(got[:, I:I + 3], value, equal_nan=True)
    assert np.array_equal(out.float().cpu().numpy()[:, :3], value, equal_nan=True)


def within(got, want, bound, x, what):
    bad = np.argwhere(~(np.abs(got - want) <= bound))
    assert not len(bad), (what, len(bad), [(x[tuple(b)], got[tuple(b)], want[tuple(b)], bound[tuple(b)]) for b in bad[:5]])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_derivative_of_every_bf16_number(act):
    x = ab.bf16_numbers()
    got = slopes(torch.from_numpy(x).bfloat16(), act).astype(np.float64)
    x = x.astype(np.float64)
    with np.errstate(over="ignore", under="ignore"):
        want = np.where(x > 1e4, 1, fr.act(np.clip(x, -1e4, 1e4), act)[1])
    within(got, want, ab.slope_bound(np.clip(x, -1e4, 1e4), want, act), x, act)


@pytest.mark.parametrize("experts,blocks", [(32, 512), (3, 64), (600, 16)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_values_in_fp32(act, experts, blocks):
    """A product of zeros with biases: gate x and up 1 at one feature of each block, up 0 at the
    others, so that the block's scale is max(|act(x)|, 2^-100) / 448."""
    G, I, K = experts, 128 * blocks, 16
    x = ab.arguments(8 * (-(-G * blocks // 8)), G)[:G * blocks].reshape(G, blocks)
    bias = torch.zeros((G, 2, blocks, 128))
    at = torch.arange(blocks) * 37 % 128
    bias[:, 0] = torch.from_numpy(ab.arguments(G * I, 1).reshape(G, blocks, 128).clip(-80, 80))
    bias[:, 0, torch.arange(blocks), at], bias[:, 1, torch.arange(blocks), at] = torch.from_numpy(x), 1.0
    zeros = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype, device="cuda")      # noqa: E731
    q, qs = mx.alloc_fp8_rows_f32_outputs(G, I)
    offs = torch.arange(G + 1, dtype=torch.int32, device="cuda")
    ws = zeros(max(16, mx.mxfp4_fp8_gated_gemm_workspace(G, G, I, K)))
    mx.mxfp4_fp8_gated_gemm(zeros(G, K), zeros(G, 1, dtype=torch.float32), zeros(G, 2, I, K),
                            zeros(G, 2, blocks, 1, dtype=torch.float32), offs, q=q, q_scales=qs,
                            bias=bias.view(G, 2 * I).cuda(), workspace=ws, act=act)
    x = x.astype(np.float64)
    value = np.abs(fr.act(x, act)[0])
    got = qs.cpu().double().numpy() * 448
    # (the division by 448 rounds once)
    within(got, np.maximum(value, 2.0 ** -100), ab.value_bound(x, value, act) + ab.U * np.maximum(got, value), x, act)

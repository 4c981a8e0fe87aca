"""The feed-forward calls once more into buffers that hold something else: every live row has to
be written again, on one stream, on others and on two at once; their E4M3 rows are the dispatch's;
and a fused layer's plan that held other tokens before."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

from test_gpu_ffn import Block

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import expert_layer  # noqa: E402


def live(b):
    """The outputs' live rows, and the biases' gradients."""
    return [t[:b.M] if len(t) == b.M_cap else t for t in b.outputs()]


def clear(b, byte):
    """Every output and the workspace, to a byte that no call leaves everywhere."""
    for t in (b.y, b.h, b.q, b.qs, b.dh, b.dq, b.dqs, b.act, b.dx, b.db1, b.db2, b.dy, b.dys, b.ws):
        t.view(torch.uint8).fill_(byte)


COUNTS = [[3, 0, 2], [60, 0, 33, 7], [300, 41], [700, 900]]


@pytest.mark.parametrize("counts", COUNTS)
def test_cleared_outputs_get_the_same_bits(counts):
    b = Block(counts, 528, 384, seed=10)
    b.run()
    want = live(b)
    for byte in (0xFF, 0x00, 0x5A):
        clear(b, byte)
        b.run()
        for got, exp in zip(live(b), want):
            assert torch.equal(got, exp), byte


@pytest.mark.parametrize("counts", COUNTS)
def test_cleared_outputs_on_another_stream(counts):
    b = Block(counts, 528, 384, seed=5)
    b.run()
    want = live(b)
    side = torch.cuda.Stream()
    for byte in (0xFF, 0x5A):
        clear(b, byte)
        side.wait_stream(torch.cuda.current_stream())
        b.run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for got, exp in zip(live(b), want):
            assert torch.equal(got, exp), byte


def test_cleared_outputs_of_two_calls_at_once():
    """Two blocks on two streams, each with buffers of its own, large ones and small ones."""
    blocks = [Block(c, 528, 384, seed=7 + i) for i, c in enumerate(COUNTS)]
    want = []
    for b in blocks:
        b.run()
        want.append(live(b))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for byte in (0xFF, 0x00, 0x5A):
        for i, j in ((0, 1), (1, 2), (2, 3), (3, 0)):
            for b in (blocks[i], blocks[j]):
                clear(b, byte)
            torch.cuda.synchronize()
            for b, s in zip((blocks[i], blocks[j]), streams):
                b.run(stream=s)
            torch.cuda.synchronize()
            for n in (i, j):
                for got, exp in zip(live(blocks[n]), want[n]):
                    assert torch.equal(got, exp), (byte, n)


def bf16_rows(M, N, seed):
    """Rows from the smallest to the largest BF16 numbers, zeros and zero blocks among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g) * torch.exp(2 * torch.randn(M, N, generator=g))
    x *= torch.exp2(torch.randint(-130, 120, (M, -(-N // 128)), generator=g).float()).repeat_interleave(128, 1)[:, :N]
    x[torch.rand(M, N, generator=g) < 0.1] = 0
    x[0, :min(N, 128)] = 0
    x = x.clamp(-3e38, 3e38).bfloat16()
    x[-1, 0] = torch.finfo(torch.bfloat16).max
    return x.cuda()


def quantized(x):
    """The dispatch's quantizer on all rows."""
    q, s = mx.alloc_fp8_rows_f32_outputs(*x.shape)
    mx.mxfp4_bf16_to_fp8_rows_f32(x, q, s, torch.tensor([0, len(x)], dtype=torch.int32, device="cuda"))
    return q, s


@pytest.mark.parametrize("M,N", [(5, 16), (77, 1360), (200, 528), (1000, 2048)])
def test_rows_gradient_has_the_dispatch_bytes(M, N):
    x = bf16_rows(M, N, M)
    q, s = mx.alloc_fp8_rows_f32_outputs(M, N)
    mx.mxfp4_act_rows_backward(x, None, torch.tensor([0, M // 3, M], dtype=torch.int32, device="cuda"), q=q, q_scales=s)
    for got, want in zip((q, s), quantized(x)):
        assert torch.equal(got, want)


def one_products(M, G, parts, I, value):
    """Operands of products that are all `value` (1 or 0) exactly."""
    K = 16
    a, w = torch.zeros((M, K), dtype=torch.uint8, device="cuda"), torch.zeros((G, parts, I, K), dtype=torch.uint8, device="cuda")
    if value:
        a[:, 0], w[..., 0] = 0x38, 0x38
    return a, torch.ones((M, 1), device="cuda"), w, torch.ones((G, parts, -(-I // 128), 1), device="cuda")


@pytest.mark.parametrize("M,I", [(3, 16), (7, 272), (40, 2048), (130, 1040)])
def test_gated_product_has_the_dispatch_bytes(M, I):
    """Products of zero with a bias for each row's expert: out = gate, a BF16 number (but for a
    negative zero, which zero plus the bias makes positive)."""
    x = bf16_rows(M, I, I)
    bias = torch.cat([x.float(), torch.ones_like(x, dtype=torch.float32)], 1)
    q, s = mx.alloc_fp8_rows_f32_outputs(M, I)
    ws = torch.empty(max(16, mx.mxfp4_fp8_gated_gemm_workspace(M, M, I, 16)), dtype=torch.uint8, device="cuda")
    mx.mxfp4_fp8_gated_gemm(*one_products(M, M, 2, I, 0), torch.arange(M + 1, dtype=torch.int32, device="cuda"), q=q,
                            q_scales=s, bias=bias, workspace=ws, act="none")
    for got, want in zip((q, s), quantized(x + 0.0)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("M,I", [(3, 128), (50, 2048), (600, 1024), (4000, 1152)])
def test_gated_gradient_has_the_dispatch_bytes(M, I):
    """Products of one: dh = [up, gate]."""
    x = bf16_rows(M, 2 * I, I)
    a, sa, w, sw = one_products(M, 1, 1, I, 1)
    q, s = mx.alloc_fp8_rows_f32_outputs(M, 2 * I)
    ws = torch.empty(max(16, mx.mxfp4_fp8_gated_gemm_backward_workspace(1, M, I, 16)), dtype=torch.uint8, device="cuda")
    mx.mxfp4_fp8_gated_gemm_backward(a, sa, w[:, 0], sw[:, 0], x, torch.tensor([0, M], dtype=torch.int32, device="cuda"),
                                     dq=q, dq_scales=s, workspace=ws, act="none")
    for got, want in zip((q, s), quantized(torch.cat([x[:, I:], x[:, :I]], 1))):
        assert torch.equal(got, want)


def test_fused_plan_of_more_tokens():
    """The same bits as with a plan of their own, whatever a call with more tokens left in it."""
    layer = expert_layer.random_layer(6, 256, 256, 3, seed=5, fused=True)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dout = (torch.randn(70, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    b = layer.plan(70)
    for n in (70, 33, 1, 70, 0):
        own = layer.plan(n)
        for keep in (False, True):
            want = layer.forward(x[:n], own, keep=keep).clone()
            got = layer.forward(x[:n], b, keep=keep)
            assert got.shape == (n, 256) and torch.equal(got, want)
        for got, want in zip(layer.backward(dout[:n], b), layer.backward(dout[:n], own)):
            assert torch.equal(got, want)
        if n:
            for got, want in zip(layer.weight_gradients(x[:n], b), layer.weight_gradients(x[:n], own)):
                assert got.isfinite().all() and torch.equal(got, want)


def test_dense_block_plan_used_again():
    """A plan that held another call's rows gives the bits of a new one."""
    r = lambda *s: torch.randn(s, device="cuda", generator=torch.Generator(device="cuda").manual_seed(sum(s)))      # noqa: E731
    block = expert_layer.FeedForward(r(512, 400) / 20, r(400, 256) / 16, 0.3 * r(512), 0.3 * r(400))
    b = block.plan(50)
    for i in range(3):
        x, dout = (r(50 + 50 * i + j, 400)[:50].bfloat16() for j in range(2))
        own = block.plan(50)
        assert np.array_equal(block.forward(x, b).float().cpu(), block.forward(x, own).float().cpu())
        for got, want in zip(block.backward(dout, b), block.backward(dout, own)):
            assert torch.equal(got, want)

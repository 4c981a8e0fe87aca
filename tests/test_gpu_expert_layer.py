"""The expert layer of examples/expert_layer.py: against a float64 layer, on a side stream,
and captured into a graph.

Both products quantize their activations to E4M3 (relative rounding error at most 2^-4 of an
element, 2^-4 / sqrt(3) / 1.4 or 0.026 in the mean), so over all outputs the 2-norm of the
error is about sqrt(2) 0.026 = 0.037 of the result's; the bound is 0.06.  The backward chain
quantizes two gradients more and multiplies by the forward's activations: 0.09.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402
import expert_layer  # noqa: E402
import moe_ref as ref  # noqa: E402


def weights64(q, s):
    nb, kb = torch.arange(q.shape[1]) // 128, torch.arange(q.shape[2]) // 128
    return torch.from_numpy(ref.e4m3(q.cpu().numpy())) * s.cpu().double()[:, nb][:, :, kb]


def reference(layer, x, ids, w, shared=None):
    """float64 output of the layer for the GPU's own choice of experts and weights."""
    up, down = weights64(layer.up, layer.up_s), weights64(layer.down, layer.down_s)
    out = shared.double() if shared is not None else torch.zeros(x.shape, dtype=torch.float64)
    for t in range(x.shape[0]):
        for j in range(layer.k):
            e = int(ids[t, j])
            if e >= 0:
                h = up[e] @ x[t].double()
                a = torch.nn.functional.silu(h[:layer.I]) * h[layer.I:]
                out[t] += float(w[t, j]) * (down[e] @ a)
    return out


@pytest.mark.parametrize("T,E,H,I,k,ng,tg", [(33, 8, 256, 128, 2, 1, 1), (1, 16, 400, 144, 4, 4, 2), (70, 12, 528, 256, 3, 1, 1)])
def test_layer_forward(T, E, H, I, k, ng, tg):
    layer = expert_layer.random_layer(E, H, I, k, ng, tg, seed=T)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    shared = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    mask = (torch.arange(T, device="cuda") % 5 != 2).to(torch.uint8)
    b = layer.plan(T)
    out = layer.forward(x, b, row_mask=mask, shared=shared)
    want = reference(layer, x.cpu(), b["ids"].cpu(), b["w"].cpu(), shared.cpu())
    err = (out.cpu().double() - want).norm() / want.norm()
    assert err <= 0.06, err
    dead = (mask == 0).cpu()
    assert torch.equal(out.cpu()[dead], shared.cpu()[dead])        # a masked token gets the base alone
    # the choice itself
    logits = b["logits"].double().cpu().numpy()
    rids, rw, gap = ref.route(logits, "sigmoid", k, bias=layer.bias.double().cpu().numpy(), row_mask=mask.cpu().numpy(),
                              n_group=ng, topk_group=tg, group_best=min(2, E // ng), scale=2.5)
    sure = gap >= 2.0 ** -14
    assert np.array_equal(b["ids"].cpu().numpy()[sure], rids[sure])


def test_layer_backward():
    layer = expert_layer.random_layer(6, 256, 128, 2, seed=3)
    T = 40
    g = torch.Generator(device="cuda").manual_seed(8)
    x, dout = (torch.randn(T, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    b = layer.plan(T)
    layer.forward(x, b)
    dx, dlogits = layer.backward(dout, b)
    up, down = weights64(layer.up, layer.up_s), weights64(layer.down, layer.down_s)
    ids = b["ids"].cpu().long()
    xr = x.cpu().double().requires_grad_()
    lr = b["logits"].double().cpu().requires_grad_()
    w = torch.sigmoid(lr).gather(1, ids)
    w = 2.5 * w / (w.sum(1, keepdim=True) + 1e-20)
    out = []
    for t in range(T):
        rows = []
        for j in range(layer.k):
            h = up[ids[t, j]] @ xr[t]
            rows.append(w[t, j] * (down[ids[t, j]] @ (torch.nn.functional.silu(h[:layer.I]) * h[layer.I:])))
        out.append(sum(rows))
    loss = (torch.stack(out) * dout.cpu().double()).sum()
    gx, gl = torch.autograd.grad(loss, (xr, lr))
    for got, want in ((dx, gx), (dlogits, gl)):
        err = (got.cpu().double() - want).norm() / want.norm()
        assert err <= 0.09, err


def test_mxfp4_path_of_the_framework():
    """Routed tokens through the MXFP4 path: dispatch, FP8 rows, UE8M0-scaled product."""
    T, E, H, N, k = 50, 4, 512, 256, 2
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    ids, w = mx.alloc_route_outputs(T, k)
    mx.mxfp4_route_topk(torch.randn(T, E, generator=g, device="cuda"), ids, w)
    offs, pos, ws = mx.alloc_expert_map_outputs(T, k, E)
    mx.mxfp4_expert_map(ids, offs, pos, ws)
    codes, scales = mx.alloc_quantize_outputs(T * k, H)
    mx.mxfp4_dispatch_rows(x, pos, codes, scales)
    # the same rows gathered first and quantized then
    xr = torch.empty((T * k, H), dtype=torch.bfloat16, device="cuda")
    xr[pos.view(-1).long()] = x.repeat_interleave(k, 0)
    c2, s2 = mx.alloc_quantize_outputs(T * k, H)
    mx.mxfp4_quantize_rows(xr, c2, s2, offs)
    assert torch.equal(codes, c2) and torch.equal(scales, s2)
    y, ys = mx.alloc_rows_outputs(T * k, H)
    mx.mxfp4_to_fp8_rows(codes, scales, y, ys, offs)
    wq = torch.randint(0, 0x7F, (E, N, H), dtype=torch.uint8, device="cuda", generator=g)
    wqs = torch.full((E, N, H // 128), 120, dtype=torch.uint8, device="cuda")
    out = torch.empty((T * k, N), dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_fp8_grouped_gemm(y, ys, wq, wqs, out, offs)
    # and the FP32-scaled product on the same numbers: power-of-two scales, so equal but for
    # the two products' FP32 sums (both within 2^-8 of the value after BF16 rounding)
    out2 = torch.empty_like(out)
    mx.mxfp4_fp8_block_gemm(y, torch.exp2(ys.float() - 127), wq,
                            torch.full((E, N // 128, H // 128), 2.0 ** -7, device="cuda"), out2, offs)
    a, b = out.double(), out2.double()
    assert (a - b).norm() <= 2.0 ** -8 * a.norm()
    back = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_combine_rows(out, pos, back, weights=w)
    assert torch.isfinite(back).all()


def test_layer_on_a_side_stream_and_repeated():
    layer = expert_layer.random_layer(16, 512, 256, 4, seed=1)
    x = torch.randn(300, 512, device="cuda").bfloat16()
    b = layer.plan(300)
    first = layer.forward(x, b).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = None
    with torch.cuda.stream(side):
        c = layer.plan(300)
        for _ in range(3):
            layer.forward(x, c)
    side.synchronize()
    assert torch.equal(first, c["out"]) and torch.equal(b["pos"], c["pos"])
    for _ in range(3):                            # the same bits every time
        assert torch.equal(layer.forward(x, b), first)


@pytest.mark.parametrize("T", [5, 700])
def test_calls_captured_into_a_graph(T):
    """Routing to combine in one graph, replayed on new inputs between eager calls; every
    replay equals the eager result."""
    E, H, N, k = 24, 512, 256, 4
    g = torch.Generator(device="cuda").manual_seed(T)
    wq, ws_ = expert_layer.quantize_weights(torch.randn(E, N, H, generator=g, device="cuda"))

    def buffers():
        ids, w = mx.alloc_route_outputs(T, k)
        offs, pos, ws = mx.alloc_expert_map_outputs(T, k, E)
        q, s = mx.alloc_fp8_rows_f32_outputs(T * k, H)
        y, out, dy, dw, dl = (torch.zeros(z, dtype=d, device="cuda") for z, d in
                              (((T * k, N), torch.bfloat16), ((T, N), torch.bfloat16), ((T * k, N), torch.bfloat16),
                               ((T, k), torch.float32), ((T, E), torch.float32)))
        return ids, w, offs, pos, ws, q, s, y, out, dy, dw, dl

    def run(x, logits, b):
        ids, w, offs, pos, ws, q, s, y, out, dy, dw, dl = b
        mx.mxfp4_route_topk(logits, ids, w, score="sigmoid")
        mx.mxfp4_expert_map(ids, offs, pos, ws)
        mx.mxfp4_dispatch_fp8_rows(x, pos, q, s)
        mx.mxfp4_fp8_block_gemm(q, s, wq, ws_, y, offs)
        mx.mxfp4_combine_rows(y, pos, out, weights=w)
        mx.mxfp4_combine_rows_backward(out, y, pos, w, dy, dw)
        mx.mxfp4_route_topk_backward(logits, ids, dw, dl, score="sigmoid")

    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    fixed, eager = buffers(), buffers()
    run(x, logits, fixed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(x, logits, fixed)
    for _ in range(4):
        x.copy_(torch.randn(T, H, generator=g, device="cuda").bfloat16())
        logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
        graph.replay()
        run(x, logits, eager)
        torch.cuda.synchronize()
        for u, v in zip(fixed, eager):
            if u is not fixed[4]:                 # (the map's workspace)
                n = u if u.shape[0] != T * k else u[:int(fixed[2][-1])]
                m = v if v.shape[0] != T * k else v[:int(fixed[2][-1])]
                assert torch.equal(n, m)

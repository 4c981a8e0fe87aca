"""The feed-forward calls in the layers of examples/expert_layer.py: a fused expert layer and a
dense block, their outputs and all their gradients against float64 and differences.

Every product quantizes its activations to E4M3 (relative rounding error at most 2^-4 of an
element, 0.026 in the mean, test_gpu_expert_layer), so the forward's error is about sqrt(2)
0.026 = 0.037 of the result's 2-norm (bound 0.06) and the gradients', with two quantized
gradients more, below 0.09.  The weights' gradients quantize both operands of one more product.
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

import expert_layer  # noqa: E402
from test_gpu_expert_layer import reference, weights64  # noqa: E402


def close(got, want, bound):
    err = (got.cpu().double() - want).norm() / want.norm()
    assert err <= bound, (err, bound)


@pytest.mark.parametrize("T,E,H,I,k,ng,tg", [(33, 8, 256, 128, 2, 1, 1), (1, 16, 400, 256, 4, 4, 2), (70, 12, 528, 256, 3, 1, 1)])
@pytest.mark.parametrize("keep", [True, False])
def test_fused_forward(T, E, H, I, k, ng, tg, keep):
    layer = expert_layer.random_layer(E, H, I, k, ng, tg, seed=T, fused=True)
    g = torch.Generator(device="cuda").manual_seed(7)
    x, shared = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    mask = (torch.arange(T, device="cuda") % 5 != 2).to(torch.uint8)
    b = layer.plan(T + 3)                         # (a plan serves fewer tokens)
    out = layer.forward(x, b, row_mask=mask, shared=shared, keep=keep)
    close(out, reference(layer, x.cpu(), b["ids"].cpu(), b["w"].cpu(), shared.cpu()), 0.06)


def test_fused_gradients():
    layer = expert_layer.random_layer(6, 256, 256, 2, seed=3, fused=True)
    T = 90
    g = torch.Generator(device="cuda").manual_seed(8)
    x, dout = (torch.randn(T, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    mask = (torch.arange(T, device="cuda") % 7 != 3).to(torch.uint8)
    b = layer.plan(T)
    layer.forward(x, b, row_mask=mask)
    dx, dlogits = layer.backward(dout, b)
    dw_up, dw_down = layer.weight_gradients(x, b)
    up, down = (weights64(q, s).requires_grad_() for q, s in ((layer.up, layer.up_s), (layer.down, layer.down_s)))
    ids = b["ids"].cpu().long()
    live = (ids >= 0).all(1)
    xr = x.cpu().double().requires_grad_()
    lr = b["logits"].double().cpu().requires_grad_()
    w = torch.sigmoid(lr).gather(1, ids.clamp_min(0))
    w = 2.5 * w / (w.sum(1, keepdim=True) + 1e-20)
    loss = 0.0
    for t in live.nonzero()[:, 0].tolist():
        for j in range(layer.k):
            h = up[ids[t, j]] @ xr[t]
            y = down[ids[t, j]] @ (torch.nn.functional.silu(h[:layer.I]) * h[layer.I:])
            loss = loss + w[t, j] * (y @ dout[t].cpu().double())
    gx, gl, gu, gd = torch.autograd.grad(loss, (xr, lr, up, down))
    for got, want in ((dx, gx), (dlogits, gl), (dw_up, gu), (dw_down, gd)):
        close(got, want, 0.09)


def test_fused_against_unfused():
    """The same layer with the activation in plain torch: within both forms' roundings."""
    a, f = (expert_layer.random_layer(8, 512, 256, 2, seed=5, fused=fused) for fused in (False, True))
    x = torch.randn(130, 512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    close(f.forward(x, f.plan(130)), a.forward(x, a.plan(130)).cpu().double(), 0.04)


def dense(H, I, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")     # noqa: E731
    return expert_layer.FeedForward(r(2 * I, H) / H ** 0.5, r(H, I) / I ** 0.5, 0.3 * r(2 * I), 0.3 * r(H)), g


@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (50, 528, 256), (300, 400, 384)])
def test_dense_block(T, H, I):
    block, g = dense(H, I, T)
    x, res, dout = (torch.randn(T, H, generator=g, device="cuda").bfloat16() for _ in range(3))
    b = block.plan(T)
    y = block.forward(x, b, residual=res)
    dx, db_up, db_down = block.backward(dout, b)
    up, down = weights64(block.up, block.up_s)[0], weights64(block.down, block.down_s)[0]
    v = [t.cpu().double().requires_grad_() for t in (x, block.b_up, block.b_down)]

    def f(x, b_up, b_down):
        h = x @ up.T + b_up
        return (torch.nn.functional.silu(h[:, :I]) * h[:, I:]) @ down.T + b_down

    want = f(*v)
    close(y.cpu().double() - res.cpu().double(), want.detach(), 0.06)
    weight = dout.cpu().double()
    grads = torch.autograd.grad((want * weight).sum(), v)
    for got, exp, bound in ((dx, grads[0], 0.09), (db_up, grads[1], 0.09), (db_down, grads[2], 1e-5)):
        close(got, exp, bound)
    # a difference of the float64 block along the gradient that came out
    step = 1e-5 * dx.cpu().double() / dx.cpu().double().norm()
    args = [t.detach() for t in v[1:]]
    diff = ((f(v[0].detach() + step, *args) - f(v[0].detach() - step, *args)) * weight).sum() / 2e-5
    assert abs(diff - dx.cpu().double().norm()) <= 0.09 * abs(diff)


def test_fused_layer_in_a_graph():
    """Captured once; every replay on new tokens as the eager call, with eager work between."""
    layer = expert_layer.random_layer(8, 512, 256, 2, seed=4, fused=True)
    T = 20
    x = torch.randn(T, 512, device="cuda").bfloat16()
    b = layer.plan(T)
    layer.forward(x, b, keep=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(x, b, keep=False)
    for i in range(4):
        x.copy_(torch.randn(T, 512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)).bfloat16())
        graph.replay()
        got = out.clone()
        torch.cuda.synchronize()
        other = layer.plan(T)
        assert np.array_equal(got.float().cpu().numpy(), layer.forward(x, other, keep=False).float().cpu().numpy()), i

"""Routing where FP32 loses most: confident experts, scores far below the largest, rows with
NaN and infinities beside rows without choices.

In units of u = 2^-24, with an exponential good to 3 u (the instruction's unit in the last
place and one rounding): a sigmoid score is good to 5 u (a sum, a division) and a weight
without renormalisation to 6 u (the scale); a softmax score adds the sum of the row, at most 8
u for the sizes here (runs of at most 4, then at most 6 levels of pairs, less the terms' own 3
u, which they share), and one division: 18 u.  A renormalised weight is a quotient of two such
numbers (the second a sum of at most 16 in 4 or 6 levels): 40 u.  A sigmoid's derivative
e / (1 + e)^2 is good to 9 u, what it is multiplied by to about 3 k + 20 u of the magnitudes
it is made of: 2^-17 of those for the k here.
"""
from __future__ import annotations

import numpy as np
import pytest

import moe_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402

U = 2.0 ** -24


def route(l, k, **kw):
    ids, w = mx.alloc_route_outputs(l.shape[0], k)
    mx.mxfp4_route_topk(l.cuda(), ids, w, **kw)
    return ids.cpu().numpy(), w.cpu().numpy()


def backward(l, ids, dw, **kw):
    dl = torch.full_like(l, 77.0, device="cuda")
    mx.mxfp4_route_topk_backward(l.cuda(), ids.cuda(), dw.cuda(), dl, **kw)
    return dl.double().cpu().numpy()


def sigmoid_gradient(l, ids, dw, renorm, scale):
    """dlogits and the magnitudes it is made of, the derivative as e / (1 + e)^2, e = exp(-|l|)."""
    e = np.exp(-np.abs(l))
    s, der = np.where(l < 0, e, 1) / (1 + e), e / (1 + e) ** 2
    sj, dj = np.take_along_axis(s, ids, 1), np.take_along_axis(der, ids, 1)
    if renorm:
        D = sj.sum(1, keepdims=True) + 1e-20
        ds = scale * (dw - (dw * sj).sum(1, keepdims=True) / D) / D
        mag = abs(scale) * (np.abs(dw) + (np.abs(dw) * sj).sum(1, keepdims=True) / D) / D
    else:
        ds, mag = scale * dw, abs(scale * dw)
    out, big = np.zeros_like(l), np.zeros_like(l)
    np.put_along_axis(out, ids, ds * dj, 1)
    np.put_along_axis(big, ids, mag * dj, 1)
    return out, big


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k,f32", [(16, 4, True), (256, 8, True), (60, 6, False), (300, 8, True), (64, 20, True)])
def test_sigmoid_gradient_of_confident_experts(E, k, f32, renorm):
    T = 64
    g = torch.Generator().manual_seed(E + k)
    size = torch.tensor([5.0, 10.0, 17.0, 30.0, 60.0])[torch.randint(0, 5, (T, E), generator=g)]
    l = size * (torch.randint(0, 2, (T, E), generator=g) * 2 - 1) + torch.randn(T, E, generator=g) * 0.5
    l = l if f32 else l.bfloat16()
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    dw = torch.randn(T, k, generator=g)
    got = backward(l, ids, dw, score="sigmoid", renorm=renorm, scale=2.5)
    want, mag = sigmoid_gradient(l.double().numpy(), ids.numpy().astype(np.int64), dw.double().numpy(), renorm, 2.5)
    assert np.all(np.abs(got - want) <= 2.0 ** -17 * mag + (0 if f32 else 2.0 ** -8) * np.abs(want) + 1e-37)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(8, 8), (16, 16), (64, 8), (64, 10)])       # both kernels
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_weights_far_below_the_largest_score(score, E, k, renorm):
    """Chosen experts down to e^-80 of the best: their weights to FP32's precision."""
    T = 500
    g = torch.Generator().manual_seed(E * k)
    l = torch.full((T, E), -85.0)
    l[:, :k] = -80 * torch.rand(T, k, generator=g)
    l = l.gather(1, torch.rand(T, E, generator=g).argsort(1))
    ids, w = route(l, k, score=score, renorm=renorm, scale=1.25)
    want = ref.weights_of(ref.scores(l.double().numpy(), score), ids.astype(np.int64), renorm, 1.25)
    bound = 40 * U if renorm else 18 * U if score == "softmax" else 6 * U
    assert np.all(np.abs(w - want) <= bound * want + 1e-37), np.abs(w / want - 1).max() / U


@pytest.mark.parametrize("E,k", [(32, 4), (300, 20)])                         # 16 lanes and a wave per token
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_rows_without_a_choice_is_zero(score, E, k):
    """Whatever their logits are: NaN, infinities, the type's lowest value."""
    T = 12
    g = torch.Generator().manual_seed(E)
    l = torch.randn(T, E, generator=g)
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    dw = torch.randn(T, k, generator=g)
    clean = backward(l, ids, dw, score=score)
    odd = [(1, torch.nan), (3, torch.inf), (5, -torch.inf), (6, torch.finfo(torch.float32).min)]
    for t, v in odd:
        l[t] = v
        ids[t] = -1
    l[8, 5], ids[8], dw[8] = torch.nan, E + 3, torch.nan
    got = backward(l, ids, dw, score=score)
    none = [t for t, _ in odd] + [8]
    assert (got[none] == 0).all()
    rest = [t for t in range(T) if t not in none]
    assert np.array_equal(got[rest], clean[rest])


def test_nan_logits_of_the_gradient():
    """Under softmax every score of such a row is NaN; a sigmoid's gradient is of the chosen alone."""
    T, E, k = 6, 40, 4
    g = torch.Generator().manual_seed(2)
    l = torch.randn(T, E, generator=g)
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    dw = torch.randn(T, k, generator=g)
    clean = {s: backward(l, ids, dw, score=s) for s in ("softmax", "sigmoid")}
    free = [e for e in range(E) if e not in ids[2].tolist()]
    l[2, free[0]], l[2, free[1]] = torch.nan, torch.inf
    rest = [0, 1, 3, 4, 5]
    got = backward(l, ids, dw, score="softmax")
    assert np.isnan(got[2]).all() and np.array_equal(got[rest], clean["softmax"][rest])
    got = backward(l, ids, dw, score="sigmoid")
    assert np.array_equal(got, clean["sigmoid"])

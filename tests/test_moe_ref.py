"""Checks of the 64-bit references themselves (CPU): gradients against differences, the map
and the selection against their definitions slot by slot."""
import math

import numpy as np
import pytest

import moe_ref as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(5)
    T, E, k = 4, 9, 3
    l = rng.normal(size=(T, E))
    ids = ref.route(l, score, k, renorm=renorm, scale=1.7)[0]
    dw = rng.normal(size=(T, k))
    grad, mag = ref.route_backward(l, ids, dw, score, renorm, 1.7)
    assert np.all(np.abs(grad) <= mag + 1e-15)
    h = 1e-6
    for e in range(E):
        d = np.zeros((T, E))
        d[:, e] = h
        hi = (dw * ref.weights_of(ref.scores(l + d, score), ids, renorm, 1.7)).sum(1)
        lo = (dw * ref.weights_of(ref.scores(l - d, score), ids, renorm, 1.7)).sum(1)
        # central difference: h^2 f''' / 6 and 1e-16 / h of rounding
        np.testing.assert_allclose((hi - lo) / (2 * h), grad[:, e], atol=1e-8)


def test_selection_by_definition():
    rng = np.random.default_rng(6)
    l = np.round(rng.normal(size=(50, 12)) * 2) / 2                # many exact ties
    bias = np.round(rng.normal(size=12)) / 4
    ids, w, _ = ref.route(l, "sigmoid", 4, bias=bias, n_group=4, topk_group=2, group_best=2)
    for t in range(50):
        c = [1 / (1 + math.exp(-v)) + b for v, b in zip(l[t], bias)]
        val = [sum(sorted(c[3 * g:3 * g + 3])[1:]) for g in range(4)]
        kept = sorted(range(4), key=lambda g: (-val[g], g))[:2]
        pool = [e for e in range(12) if e // 3 in kept]
        assert list(ids[t]) == sorted(pool, key=lambda e: (-c[e], e))[:4]
    np.testing.assert_allclose(w.sum(1), 1, rtol=1e-12)


def test_map_by_definition():
    ids = np.array([[3, 5], [-1, 3], [4, 9], [5, 3]])
    offs, pos, src = ref.expert_map(ids, 3, 3, 8)
    assert list(offs) == [0, 3, 4, 6]
    assert pos.tolist() == [[0, 4], [-1, 1], [3, -1], [5, 2]]
    assert list(src) == [0, 3, 7, 4, 1, 6]
    offs, pos, src = ref.expert_map(ids, 3, 3, 4)                   # only four rows fit
    assert list(offs) == [0, 3, 4, 4] and list(src) == [0, 3, 7, 4]
    assert pos.tolist() == [[0, -1], [-1, 1], [3, -1], [-1, 2]]


def test_e4m3_values():
    import torch
    b = np.array([i for i in range(256) if i & 0x7F != 0x7F], np.uint8)
    want = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(b), want)

"""Routing on the GPU against the 64-bit definition.

Ids are compared where the choice does not hang on FP32 rounding: every deciding gap is an
exact tie (the index decides) or at least 2^-14 of the values, eight times what the FP32
scores can be off by 2^-17 (exp with its argument's rounding |l - m| 2^-24 for |l - m| <= 32,
a sum of at most 1024 positive terms, one division).  Weights: 2^-16 of themselves (score,
sum over k, division).  Gradient: 2^-14 of the magnitudes it is summed from, and 2^-8 of
itself for BF16.
"""
from __future__ import annotations

import numpy as np
import pytest

import moe_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402

CANARY = -77


def run_route(logits, k, **kw):
    T = logits.shape[0]
    ids = torch.full((T + 1, k), CANARY, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), float(CANARY), device="cuda")
    mx.mxfp4_route_topk(logits.cuda(), ids[:T], w[:T], **kw)
    assert (ids[T:] == CANARY).all() and (w[T:] == CANARY).all()
    return ids[:T].cpu().numpy(), w[:T].cpu().numpy()


def inputs(T, E, f32, seed):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 1.5 + torch.randn(E, generator=g) * 0.5
    return l if f32 else l.bfloat16(), torch.randn(E, generator=g) * 0.1


CASES = [
    # T, E, n_group, topk_group, group_best, k, score, bias, f32
    (1, 1, 1, 1, 1, 1, "softmax", False, True),
    (1, 256, 8, 4, 2, 8, "sigmoid", True, True),
    (37, 256, 8, 4, 2, 8, "sigmoid", True, False),
    (1000, 256, 1, 1, 1, 8, "softmax", False, True),
    (5, 60, 1, 1, 1, 4, "softmax", False, False),
    (63, 61, 1, 1, 1, 61, "softmax", True, True),
    (65, 64, 64, 64, 1, 64, "sigmoid", False, True),
    (9, 160, 8, 3, 1, 6, "softmax", False, True),
    (33, 1024, 64, 5, 2, 17, "softmax", True, True),
    (33, 1023, 33, 9, 2, 64, "sigmoid", True, False),
    (17, 1000, 1, 1, 1, 3, "sigmoid", False, True),
    (70, 45, 3, 2, 2, 12, "softmax", True, False),
    (12, 30, 5, 5, 1, 30, "sigmoid", True, True),
    (3, 1020, 17, 3, 2, 5, "softmax", False, True),
    (130, 2, 2, 1, 1, 1, "softmax", False, True),
    (4100, 128, 4, 2, 2, 6, "softmax", False, True),
    (257, 12, 1, 1, 1, 3, "softmax", False, True),
    (129, 20, 4, 2, 2, 4, "sigmoid", True, False),
    (300, 384, 8, 2, 2, 16, "sigmoid", True, True),
]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case, renorm):
    T, E, ng, tg, gb, k, score, has_bias, f32 = case
    l, bias = inputs(T, E, f32, seed=E + T)
    mask = (torch.arange(T) % 7 != 3).to(torch.uint8)
    kw = dict(n_group=ng, topk_group=tg, group_best=gb, renorm=renorm, scale=1.25)
    ids, w = run_route(l, k, bias=bias.cuda() if has_bias else None, row_mask=mask.cuda(), score=score, **kw)
    rids, rw, gap = ref.route(l.double().numpy(), score, k, bias=bias.numpy() if has_bias else None,
                              row_mask=mask.numpy(), **kw)
    live = mask.numpy() != 0
    assert (ids[~live] == -1).all() and (w[~live] == 0).all()
    assert ((ids[live] >= 0) & (ids[live] < E)).all()
    assert all(len(set(r)) == k for r in ids[live])
    sure = live & (gap >= 2.0 ** -14)
    if k < 30:                                    # (long lists have a close pair in many rows)
        assert sure.sum() >= 0.8 * live.sum() - 1
    assert np.array_equal(ids[sure], rids[sure])
    # all rows: the weights that belong to the ids that were chosen
    s = ref.scores(l.double().numpy(), score)
    want = ref.weights_of(s[live], ids[live].astype(np.int64), renorm, 1.25)
    assert np.all(np.abs(w[live] - want) <= 2.0 ** -16 * np.abs(want) + 1e-37)


def test_ties_go_to_the_lower_index():
    l = torch.zeros(3, 96)
    l[1, 50:60] = 1
    l[2] = torch.tensor([1.0, 2.0] * 48)
    ids, _ = run_route(l, 8, score="softmax")
    assert ids.tolist() == [list(range(8)), list(range(50, 58)), list(range(1, 17, 2))]
    ids, _ = run_route(l, 8, score="sigmoid", n_group=4, topk_group=2, group_best=2)
    assert ids[0].tolist() == list(range(8))
    assert ids[1].tolist() == list(range(50, 58))
    assert ids[2].tolist() == list(range(1, 17, 2))
    bias = torch.zeros(60)
    bias[50] = -0.0                               # equal to +0
    ids, _ = run_route(torch.full((1, 60), -torch.inf), 60, score="softmax", bias=bias.cuda())
    assert ids[0].tolist() == list(range(60))


def test_infinities_nan_and_lowest_values():
    inf, nan, low = torch.inf, torch.nan, torch.finfo(torch.float32).min
    E = 40
    l = torch.randn(8, E, generator=torch.Generator().manual_seed(1))
    l[0] = -inf                                   # nothing is left: zero weights, valid ids
    l[1] = low                                    # the type's lowest value everywhere: uniform
    l[2, 5:] = -inf                               # fewer finite experts than choices
    l[3, 7] = nan
    l[4, 9] = inf
    l[5, ::2] = low
    l[6] = 3e38
    ids, w = run_route(l, 8, score="softmax")
    assert all(sorted(set(r)) == sorted(r) and min(r) >= 0 and max(r) < E for r in ids.tolist())
    assert ids[0].tolist() == list(range(8)) and (w[0] == 0).all()
    assert ids[1].tolist() == list(range(8)) and np.allclose(w[1], 1 / 8, rtol=2.0 ** -16)
    assert set(ids[2][:5]) == set(range(5)) and (w[2][5:] == 0).all() and abs(w[2].sum() - 1) < 2.0 ** -16
    assert ids[2][5:].tolist() == [5, 6, 7]
    assert np.isnan(w[3]).all() and np.isnan(w[4]).all()
    assert all(e % 2 == 1 for e in ids[5])
    assert ids[6].tolist() == list(range(8)) and np.allclose(w[6], 1 / 8, rtol=2.0 ** -16)
    ids, w = run_route(l, 8, score="sigmoid")
    assert all(sorted(set(r)) == sorted(r) and min(r) >= 0 and max(r) < E for r in ids.tolist())
    assert (w[0] == 0).all() and 7 not in ids[3] and ids[4][0] == 9
    assert not np.isnan(w[[0, 1, 2, 4, 5, 6, 7]]).any()
    # NaN and -inf in the bias: lower than every number, below -inf too
    bias = torch.zeros(E)
    bias[:30] = -inf
    bias[30:35] = nan
    ids, _ = run_route(torch.zeros(1, E), E, score="sigmoid", bias=bias.cuda())
    assert ids[0].tolist() == list(range(35, 40)) + list(range(30)) + list(range(30, 35))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,f32,renorm", [(1, 1, 1, True, False), (1, 256, 8, True, True), (129, 60, 4, False, True),
                                              (40, 1024, 64, True, True), (7, 1023, 3, False, False),
                                              (1000, 256, 8, True, True), (300, 17, 17, True, True),
                                              (4099, 96, 6, False, True), (18, 384, 10, True, False)])
def test_backward(score, T, E, k, f32, renorm):
    l, _ = inputs(T, E, f32, seed=3 * E + T)
    g = torch.Generator().manual_seed(9)
    ids = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32)
    if T > 4:
        ids[2] = -1                               # a masked row
        ids[3, 0] = E                             # an id that is none
    dw = torch.randn(T, k, generator=g)
    dl = torch.full((T + 1, E), float(CANARY), dtype=l.dtype, device="cuda")
    mx.mxfp4_route_topk_backward(l.cuda(), ids.cuda(), dw.cuda(), dl[:T], score=score, renorm=renorm, scale=2.5)
    assert (dl[T:] == CANARY).all()
    got = dl[:T].double().cpu().numpy()
    want, mag = ref.route_backward(l.double().numpy(), ids.numpy().astype(np.int64), dw.numpy(), score, renorm, 2.5)
    tol = 2.0 ** -14 * mag + (0 if f32 else 2.0 ** -8) * np.abs(want) + 1e-37
    assert np.all(np.abs(got - want) <= tol)
    if T > 4:
        assert (got[2] == 0).all()


def test_backward_against_differences():
    """The GPU gradient against central differences of the 64-bit forward (step 1e-5: h^2 of
    the third derivative below 1e-9, rounding 1e-11; the gradient's own error 2^-14)."""
    T, E, k = 3, 24, 5
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(3))
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(4))
    for score in ("softmax", "sigmoid"):
        ids, _ = run_route(l, k, score=score)
        dl = torch.empty(T, E, device="cuda")
        mx.mxfp4_route_topk_backward(l.cuda(), torch.from_numpy(ids).cuda(), dw.cuda(), dl, score=score)
        l64, at = l.double().numpy(), ids.astype(np.int64)
        _, mag = ref.route_backward(l64, at, dw.numpy(), score, True, 1.0)
        for e in range(E):
            d = np.zeros((T, E))
            d[:, e] = 1e-5
            hi = (dw.numpy() * ref.weights_of(ref.scores(l64 + d, score), at, True, 1.0)).sum(1)
            lo = (dw.numpy() * ref.weights_of(ref.scores(l64 - d, score), at, True, 1.0)).sum(1)
            assert np.all(np.abs(dl[:, e].cpu().numpy() - (hi - lo) / 2e-5) <= 2.0 ** -14 * mag[:, e] + 1e-8)


def test_backward_of_rows_with_nothing_left():
    l = torch.full((2, 32), -torch.inf)
    l[1, 3] = 0
    ids = torch.tensor([[0, 1], [3, 4]], dtype=torch.int32)
    dl = torch.empty(2, 32, device="cuda")
    mx.mxfp4_route_topk_backward(l.cuda(), ids.cuda(), torch.ones(2, 2, device="cuda"), dl, score="softmax")
    assert (dl == 0).all()

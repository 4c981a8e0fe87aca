"""The expert map, dispatch and combine on the GPU.

Map: equal to the slot-by-slot definition.  Dispatch: every byte equal to the quantizers'
definitions (MXFP4: the oracle's; FP8: the FP32 steps of the header), rows without a slot
untouched.  Combine: 2^-8 of the value (BF16 rounding) + (k + 2) 2^-24 of the sum of
magnitudes (the FP32 sum); gradients: dy bit for bit (one FP32 product, one rounding),
dweights K 2^-24 of the sum of magnitudes.
"""
from __future__ import annotations

import numpy as np
import pytest

import moe_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import block_scaled_precision_bf16tofp4row_amd as mx  # noqa: E402
import oracle  # noqa: E402

SENTINEL = -123456


def make_map(ids, G, first=0, M_cap=None, src=True):
    T, k = ids.shape
    M_cap = T * k if M_cap is None else M_cap
    offs = torch.full((G + 2,), SENTINEL, dtype=torch.int32, device="cuda")
    pos = torch.full((T + 1, k), SENTINEL, dtype=torch.int32, device="cuda")
    s = torch.full((M_cap + 1,), SENTINEL, dtype=torch.int32, device="cuda") if src else None
    ws = torch.empty(max(1, mx.mxfp4_expert_map_workspace(T, k, G) // 4), dtype=torch.int32, device="cuda")
    mx.mxfp4_expert_map(torch.as_tensor(ids, dtype=torch.int32).cuda(), offs[:G + 1], pos[:T], ws,
                        src=s[:M_cap] if src else None, first_expert=first, G=G, M_cap=M_cap)
    assert offs[G + 1] == SENTINEL and (pos[T:] == SENTINEL).all()
    return offs[:G + 1], pos[:T], s


def routed(T, k, E, seed, skew=1.0):
    g = torch.Generator().manual_seed(seed)
    pull = torch.randn(E, generator=g) * skew
    if k <= E:
        ids = (torch.rand(T, E, generator=g).log().neg().log().neg() + pull).topk(k, 1).indices.to(torch.int32)
    else:
        ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    ids[torch.rand(T, generator=g) < 0.1] = -1
    return ids


@pytest.mark.parametrize("T,k,E,first,G", [(0, 3, 4, 0, 4), (1, 1, 1, 0, 1), (1, 8, 256, 0, 256), (64, 8, 256, 32, 32),
                                           (63, 6, 64, 0, 64), (511, 8, 32, 0, 32), (512, 8, 40, 8, 16),
                                           (513, 8, 40, 8, 16), (4099, 8, 256, 0, 256), (9000, 6, 1024, 0, 1024),
                                           (20000, 2, 8, 0, 8), (70001, 8, 160, 20, 100), (40, 64, 64, 0, 63),
                                           (1025, 4, 1000, 990, 700)])
def test_map(T, k, E, first, G):
    ids = routed(T, k, E, seed=T + E)
    offs, pos, src = make_map(ids, G, first)
    roffs, rpos, rsrc = ref.expert_map(ids.numpy(), first, G, T * k)
    assert np.array_equal(offs.cpu().numpy(), roffs)
    assert np.array_equal(pos.cpu().numpy(), rpos)
    s = src.cpu().numpy()
    assert np.array_equal(s[:len(rsrc)], rsrc) and (s[len(rsrc):] == SENTINEL).all()


@pytest.mark.parametrize("T,k,M_cap", [(100, 4, 0), (100, 4, 57), (6000, 4, 9999)])
def test_map_with_too_few_rows(T, k, M_cap):
    ids = routed(T, k, 16, seed=2)
    offs, pos, src = make_map(ids, 16, 0, M_cap)
    roffs, rpos, rsrc = ref.expert_map(ids.numpy(), 0, 16, M_cap)
    assert np.array_equal(offs.cpu().numpy(), roffs) and np.array_equal(pos.cpu().numpy(), rpos)
    s = src.cpu().numpy()
    assert np.array_equal(s[:len(rsrc)], rsrc) and (s[len(rsrc):] == SENTINEL).all()


@pytest.mark.parametrize("T", [50, 5000])
def test_map_of_extreme_ids(T):
    """No slot here, all slots at one expert, ids at the ends of int32, a map without src."""
    for value, first in ((-1, 0), (7, 0), (2 ** 31 - 1, 5), (-2 ** 31, 5), (2 ** 31 - 1, 2 ** 31 - 1)):
        ids = torch.full((T, 2), value, dtype=torch.int32)
        offs, pos, _ = make_map(ids, 9, first, src=False)
        roffs, rpos, _ = ref.expert_map(ids.numpy(), first, 9, 2 * T)
        assert np.array_equal(offs.cpu().numpy(), roffs) and np.array_equal(pos.cpu().numpy(), rpos)


def bf16_rows(T, K, seed, wide=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g)
    if wide:                                      # blocks over the whole exponent range, zero blocks
        x = torch.ldexp(x, torch.randint(-140, 120, (T, 1), generator=g))
        x[torch.rand(T, K, generator=g) < 0.2] = -0.0
        if T > 2:
            x[1] = 0
    return x.bfloat16()


def bits(x):
    return x.contiguous().view(torch.int16).numpy().view(np.uint16)


SHAPES = [(1, 1, 1, 16), (3, 2, 4, 112), (70, 8, 32, 128), (5, 64, 64, 1040), (33, 6, 16, 2048), (9, 3, 8, 7168),
          (130, 2, 4, 4112), (1, 8, 256, 7168)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,k,E,K", SHAPES)
def test_dispatch_fp8(T, k, E, K, wide):
    ids = routed(T, k, E, seed=K)
    G = max(1, E - 1)                             # the last expert is elsewhere
    offs, pos, src = make_map(ids, G)
    x = bf16_rows(T, K, seed=T, wide=wide)
    cap, kb = T * k, (K + 127) // 128
    y = torch.full((cap + 1, K), 0xA5, dtype=torch.uint8, device="cuda")
    ys = torch.full((cap + 1, kb), -5.0, device="cuda")
    mx.mxfp4_dispatch_fp8_rows(x.cuda(), pos, y[:cap], ys[:cap])
    q, s = ref.fp8_rows_f32(x)
    n = int(offs[-1])
    token = src[:n].cpu().numpy() // k
    assert np.array_equal(y[:n].cpu().numpy(), q[token])
    assert np.array_equal(ys[:n].cpu().numpy().view(np.uint32), s[token].view(np.uint32))
    assert (y[n:] == 0xA5).all() and (ys[n:] == -5).all()
    # rows in expert order already
    xr = torch.full((cap, K), 1.0, dtype=torch.bfloat16, device="cuda")
    xr[:n] = x.cuda()[torch.from_numpy(token).cuda()]
    y2 = torch.full((cap + 1, K), 0xA5, dtype=torch.uint8, device="cuda")
    ys2 = torch.full((cap + 1, kb), -5.0, device="cuda")
    mx.mxfp4_bf16_to_fp8_rows_f32(xr, y2[:cap], ys2[:cap], offs)
    assert torch.equal(y2, y) and torch.equal(ys2, ys)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,k,E,K", [(1, 1, 1, 32), (3, 2, 4, 96), (70, 8, 32, 128), (5, 64, 64, 1056),
                                     (33, 6, 16, 2048), (9, 3, 8, 7168)])
def test_dispatch_mxfp4(T, k, E, K, wide):
    ids = routed(T, k, E, seed=K)
    G = max(1, E - 1)
    offs, pos, src = make_map(ids, G)
    x = bf16_rows(T, K, seed=T, wide=wide)
    cap = T * k
    codes = torch.full((cap + 1, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    sc = torch.full((cap + 1, K // 32), 0xA5, dtype=torch.uint8, device="cuda")
    mx.mxfp4_dispatch_rows(x.cuda(), pos, codes[:cap], sc[:cap])
    c, s = oracle.quantize_rows(bits(x), rows=T)
    n = int(offs[-1])
    token = src[:n].cpu().numpy() // k
    assert np.array_equal(codes[:n].cpu().numpy(), c[token])
    assert np.array_equal(sc[:n].cpu().numpy(), s[token])
    assert (codes[n:] == 0xA5).all() and (sc[n:] == 0xA5).all()


@pytest.mark.parametrize("K", [912, 928, 944, 960, 976, 992, 1008, 1936, 3024, 7152])
def test_partial_last_block_of_whole_waves(K):
    """Rows whose blocks fill whole waves and whose last block is partial: its lanes without
    elements take part in the block's maximum."""
    test_dispatch_fp8(37, 3, 8, K, False)
    if K % 32 == 0:
        test_dispatch_mxfp4(37, 3, 8, K, False)


def test_positions_outside_the_output_are_skipped():
    T, k, K, cap = 4, 3, 128, 5
    pos = torch.tensor([[0, 5, -7], [2 ** 31 - 1, -2 ** 31, 1], [2, 6, 3], [-1, -1, 4]], dtype=torch.int32).cuda()
    x = bf16_rows(T, K, seed=0)
    y, ys = mx.alloc_fp8_rows_f32_outputs(cap, K)
    mx.mxfp4_dispatch_fp8_rows(x.cuda(), pos, y, ys)
    q, s = ref.fp8_rows_f32(x)
    token = [0, 1, 2, 2, 3]
    assert np.array_equal(y.cpu().numpy(), q[token]) and np.array_equal(ys.cpu().numpy(), s[token])
    rows = bf16_rows(cap, K, seed=1)
    out = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_combine_rows(rows.cuda(), pos, out)
    want = torch.stack([rows[0], rows[1], (rows[2].float() + rows[3].float()).bfloat16(), rows[4]])
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("weighted,based", [(True, True), (False, False), (True, False)])
@pytest.mark.parametrize("T,k,E,K", [(1, 1, 1, 8), (3, 2, 4, 104), (70, 8, 32, 512), (5, 64, 70, 1032), (33, 6, 16, 2048),
                                     (9, 9, 12, 7168), (1, 8, 64, 7168), (2100, 3, 8, 136)])
def test_combine(T, k, E, K, weighted, based):
    ids = routed(T, k, E, seed=K)
    G = max(1, E - 1)
    offs, pos, _ = make_map(ids, G)
    cap = T * k
    y = bf16_rows(cap, K, seed=3)
    y[int(offs[-1]):] = float("nan")              # rows without a slot are not read
    g = torch.Generator().manual_seed(4)
    w = torch.randn(T, k, generator=g)
    base = bf16_rows(T, K, seed=5)
    p = pos.cpu().numpy()
    w[torch.from_numpy(p < 0)] = float("nan")     # nor are the weights of choices without a row
    out = torch.full((T + 1, K), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.mxfp4_combine_rows(y.cuda(), pos, out[:T], weights=w.cuda() if weighted else None,
                          base=base.cuda() if based else None)
    yv = y.double().numpy()
    want = base.double().numpy().copy() if based else np.zeros((T, K))
    mag = np.abs(want)
    for j in range(k):
        at = np.nonzero(p[:, j] >= 0)[0]
        term = yv[p[at, j]] * (w[at, j].double().numpy()[:, None] if weighted else 1.0)
        want[at] += term
        mag[at] += np.abs(term)
    got = out[:T].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (k + 2) * 2.0 ** -24 * mag + 1e-38)
    assert (out[T:] == 7).all()


@pytest.mark.parametrize("T,k,E,K", [(1, 1, 1, 8), (3, 2, 4, 104), (70, 8, 32, 512), (5, 64, 70, 1032), (33, 6, 16, 2048),
                                     (9, 9, 12, 7168), (2051, 3, 8, 136), (2048, 2, 4, 520)])
def test_combine_backward(T, k, E, K):
    ids = routed(T, k, E, seed=K + 1)
    G = max(1, E - 1)
    offs, pos, src = make_map(ids, G)
    cap, n = T * k, int(offs[-1])
    y = bf16_rows(cap, K, seed=3)
    y[n:] = float("nan")
    g = torch.Generator().manual_seed(4)
    w, dout = torch.randn(T, k, generator=g), bf16_rows(T, K, seed=6)
    p = pos.cpu().numpy()
    w[torch.from_numpy(p < 0)] = float("nan")
    dy = torch.full((cap + 1, K), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((T + 1, k), 7.0, device="cuda")
    mx.mxfp4_combine_rows_backward(dout.cuda(), y.cuda(), pos, w.cuda(), dy[:cap], dw[:T])
    s = src[:n].cpu().long()
    want = (dout[s // k].float() * w.view(-1)[s][:, None]).bfloat16()
    assert torch.equal(dy[:n].cpu().view(torch.int16), want.view(torch.int16))
    assert (dy[n:] == 7).all() and (dw[T:] == 7).all()
    got = dw[:T].cpu().numpy()
    d = dout.double().numpy()
    for j in range(k):
        at = np.nonzero(p[:, j] >= 0)[0]
        term = d[at] * y.double().numpy()[p[at, j]]
        assert np.all(np.abs(got[at, j] - term.sum(1)) <= K * 2.0 ** -24 * np.abs(term).sum(1) + 1e-38)
        assert (got[p[:, j] < 0, j] == 0).all()


def test_combine_gradients_against_differences():
    """dw and dy against differences of the GPU's own forward in a linear function: exact up to
    the BF16 rounding of the two outputs (2^-8 of their sizes) and of dy."""
    T, k, K = 4, 2, 64
    ids = torch.tensor([[0, 1], [1, 2], [2, 0], [-1, 1]], dtype=torch.int32)
    offs, pos, _ = make_map(ids, 3)
    n = int(offs[-1])
    y = bf16_rows(T * k, K, seed=1).cuda()
    w = torch.randn(T, k, generator=torch.Generator().manual_seed(2)).cuda()
    dout = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    dout[:, 5] = 1.0                              # <dout, out> = the sum of column 5
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    mx.mxfp4_combine_rows_backward(dout, y, pos, w, dy, dw)

    def value(weights, rows):
        out = torch.empty((T, K), dtype=torch.bfloat16, device="cuda")
        mx.mxfp4_combine_rows(rows, pos, out, weights=weights)
        return out[:, 5].double().cpu()

    for t in range(T):
        for j in range(k):
            step = torch.zeros_like(w)
            step[t, j] = 0.5
            hi, lo = value(w + step, y), value(w - step, y)
            assert abs((hi - lo).sum() - dw[t, j].item()) <= 2.0 ** -8 * (hi.abs() + lo.abs()).sum()
    for r in range(n):
        step = torch.zeros_like(y)
        step[r, 5] = 1.0
        hi, lo = value(w, (y.float() + step.float()).bfloat16()), value(w, (y.float() - step.float()).bfloat16())
        assert abs((hi - lo).sum() / 2 - dy[r, 5].item()) <= 2.0 ** -7 * (hi.abs() + lo.abs()).sum() + 2.0 ** -8 * w.abs().max().item() * 4

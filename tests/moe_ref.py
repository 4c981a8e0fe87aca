"""Plain implementations, in 64 bits or with the stated FP32 steps, of routing, the expert
map, dispatch, the FP32-scaled product and combine (the references of test_gpu_route,
test_gpu_dispatch, test_gpu_combine and test_gpu_block_gemm)."""
from __future__ import annotations

import numpy as np
import torch


# ---- routing ---------------------------------------------------------------------------

def scores(logits: np.ndarray, score: str) -> np.ndarray:
    """float64 scores of float64 logits [T, E]: a row of -inf only gives zeros under softmax."""
    l = logits.astype(np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1 / (1 + np.exp(-l))
    m = l.max(1, keepdims=True)
    p = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    d = p.sum(1, keepdims=True)
    return np.divide(p, d, out=np.zeros_like(p), where=d != 0)


def _first_best(c, n):
    """Indices of the n largest of each row, equal values by index, NaN below every number."""
    c = np.where(np.isnan(c), -np.inf, c) if np.isnan(c).any() else c
    return np.argsort(-c, axis=1, kind="stable")[:, :n]


def route(logits, score, k, bias=None, row_mask=None, n_group=1, topk_group=1, group_best=1, renorm=True, scale=1.0):
    """ids, weights and the smallest relative gap that decided a row (groups or experts; exact
    ties, which the index decides, do not count)."""
    T, E = logits.shape
    s = scores(logits, score)
    c = s if bias is None else s + bias.astype(np.float64)
    gap = np.full(T, np.inf)

    def decided(v):
        d = v[:, :-1] - v[:, 1:]
        size = np.maximum(np.abs(v[:, :-1]), 1e-30)
        r = np.where(d > 0, d / size, np.inf)
        return r.min(1) if r.shape[1] else np.full(T, np.inf)

    if topk_group < n_group:
        per = c.reshape(T, n_group, -1)
        gv = -np.sort(-per, axis=2)[:, :, :group_best].sum(2)
        order = _first_best(gv, n_group)
        gap = np.minimum(gap, decided(np.take_along_axis(gv, order, 1)[:, :topk_group + 1]))
        keep = np.zeros((T, n_group), bool)
        np.put_along_axis(keep, order[:, :topk_group], True, 1)
        c = np.where(np.repeat(keep, E // n_group, 1), c, -np.inf)
        best = np.where(np.isneginf(c), -1e300, c)
    else:
        best = c
    order = _first_best(best, E)
    v = np.take_along_axis(best, order, 1)[:, :k + 1]
    gap = np.minimum(gap, decided(v))
    ids = order[:, :k].astype(np.int64)
    w = weights_of(s, ids, renorm, scale)
    if row_mask is not None:
        dead = row_mask == 0
        ids[dead] = -1
        w[dead] = 0
    return ids, w, gap


def weights_of(s, ids, renorm, scale):
    w = np.take_along_axis(s, ids, 1)
    return scale * w / (w.sum(1, keepdims=True) + 1e-20) if renorm else scale * w


def route_backward(logits, ids, dw, score, renorm, scale):
    """dlogits in float64, and the sum of the magnitudes it is made of (for error bounds)."""
    s = scores(logits, score)
    T, E = s.shape
    ok = (ids >= 0) & (ids < E)
    at = np.where(ok, ids, 0)
    sj = np.where(ok, np.take_along_axis(s, at, 1), 0.0)
    g = np.where(ok, dw.astype(np.float64), 0.0)
    if renorm:
        D = sj.sum(1, keepdims=True) + 1e-20
        ds = scale * (g - (g * sj).sum(1, keepdims=True) / D) / D
        mag = abs(scale) * (np.abs(g) + (np.abs(g) * sj).sum(1, keepdims=True) / D) / D
    else:
        ds, mag = scale * g, abs(scale) * np.abs(g)
    ds, mag = np.where(ok, ds, 0.0), np.where(ok, mag, 0.0)
    full, fmag = np.zeros((T, E)), np.zeros((T, E))
    for j in range(ids.shape[1]):
        r = np.nonzero(ok[:, j])[0]
        full[r, ids[r, j]] = ds[r, j]
        fmag[r, ids[r, j]] = mag[r, j]
    if score == "sigmoid":
        return full * s * (1 - s), fmag * s * (1 - s)
    return s * (full - (ds * sj).sum(1, keepdims=True)), s * (fmag + (mag * sj).sum(1, keepdims=True))


# ---- the map ---------------------------------------------------------------------------

def expert_map(ids: np.ndarray, first: int, G: int, M_cap: int):
    slots = ids.reshape(-1).astype(np.int64) - first
    lists = [np.nonzero(slots == g)[0] for g in range(G)]
    offs = np.concatenate([[0], np.cumsum([len(v) for v in lists])])
    order = np.concatenate(lists) if lists else np.zeros(0, np.int64)
    pos = np.full(slots.size, -1, np.int64)
    keep = order[:M_cap]
    pos[keep] = np.arange(len(keep))
    return np.minimum(offs, M_cap).astype(np.int64), pos.reshape(ids.shape), keep


# ---- quantization ----------------------------------------------------------------------

def bits_to_f32(b: np.ndarray) -> np.ndarray:
    return (b.astype(np.uint32) << 16).view(np.float32)


def fp8_rows_f32(x: torch.Tensor):
    """E4M3 bytes and FP32 scales of BF16 rows [T, K] on the CPU, by the FP32 steps of the
    definition: a = max(amax, 2^-100), scale a / 448, E4M3(x * (448 / a))."""
    T, K = x.shape
    kb = (K + 127) // 128
    f = torch.zeros((T, kb * 128), dtype=torch.float32)
    f[:, :K] = x.float()
    f = f.view(T, kb, 128)
    a = f.abs().amax(2, keepdim=True).clamp_min(2.0 ** -100)
    q = (f * (torch.tensor(448.0) / a)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(T, -1)[:, :K].contiguous().numpy(), (a / 448).view(T, kb).numpy()


def e4m3(b: np.ndarray) -> np.ndarray:
    """E4M3FN bytes -> float64."""
    b = b.astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where(b & 0x80, -v, v)


# ---- product ---------------------------------------------------------------------------

def block_product(a, sa, w, sw, offs):
    """float64 y and the sum of |terms|, for uint8 a [M, K], w [G, N, K] and float32 scales."""
    M, K = a.shape
    G, N, _ = w.shape
    kb = np.arange(K) // 128
    nb = np.arange(N) // 128
    av = e4m3(a) * sa.astype(np.float64)[:, kb]
    y, mag = np.zeros((M, N)), np.zeros((M, N))
    for g in range(G):
        r = slice(int(offs[g]), int(offs[g + 1]))
        if r.start < r.stop:
            wv = e4m3(w[g]) * sw[g].astype(np.float64)[nb][:, kb]
            y[r] = av[r] @ wv.T
            mag[r] = np.abs(av[r]) @ np.abs(wv).T
    return y, mag

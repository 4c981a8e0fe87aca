"""Plain float64 implementations of the feed-forward operators (the references of
test_gpu_ffn.py), with bounds on what the kernels may be off.

A product's FP32 sums are off by at most
    E = (2^-10 + (K / 128 + 4) 2^-24) sum|terms| + 2^-133
(2^-10: the matrix core's own rounding of a 64-term dot product, as test_gpu_gemm measures it,
with margin; the rest the FP32 sum over the blocks), and a bias adds one rounding.  Activations
and derivatives are good to (|x| + 8) 2^-22 of the value and of 1; their slopes are at most 1.2
and their curvatures at most 0.9 (the largest: both gelu at 0, sqrt(2 / pi); silu 0.5).
"""
from __future__ import annotations

import numpy as np
from scipy.special import expit, ndtr

import moe_ref as ref

SLOPE = 1.2
C = np.sqrt(2 / np.pi)


def act(x, name):
    """The activation and its derivative."""
    x = np.asarray(x, np.float64)
    if name == "none":
        return x, np.ones_like(x)
    if name == "relu":
        return np.maximum(x, 0), (x > 0).astype(np.float64)
    if name == "silu":
        s = expit(x)
        return x * s, s + x * s * expit(-x)
    if name == "gelu":
        return x * ndtr(x), ndtr(x) + x * np.exp(-x * x / 2) / np.sqrt(2 * np.pi)
    assert name == "gelu_tanh"
    u = 2 * C * (x + 0.044715 * x ** 3)
    s = expit(u)
    return x * s, s + x * s * expit(-u) * 2 * C * (1 + 3 * 0.044715 * x * x)


def act_error(x):
    """How far an activation may be off, relative to its value, and its derivative, absolute."""
    return (np.abs(x) + 8) * 2.0 ** -22


def product(a, sa, w, sw, offs, bias=None):
    """float64 rows and how far their FP32 sums may be off."""
    y, mag = ref.block_product(a, sa, w, sw, offs)
    err = (2.0 ** -10 + (a.shape[1] / 128 + 4) * 2.0 ** -24) * mag + 2.0 ** -133
    if bias is not None:
        b = bias.astype(np.float64)[expert_of(offs, len(a))]
        err = err + 2.0 ** -23 * (np.abs(y) + np.abs(b))
        y = y + b
    return y, err


def expert_of(offs, rows):
    return np.searchsorted(offs, np.arange(rows), side="right") - 1


def gated_h(a, sa, w, sw, offs, bias=None):
    """h = [gate, up] of weights [G, 2, I, K], and its error."""
    halves = [product(a, sa, w[:, p], sw[:, p], offs, None if bias is None else bias[:, p]) for p in range(2)]
    return np.concatenate([h[0] for h in halves], 1), np.concatenate([h[1] for h in halves], 1)


def gated_out(h, eh, name):
    """act(gate) up and its error, from h and its error."""
    n = h.shape[1] // 2
    g, u, eg, eu = h[:, :n], h[:, n:], eh[:, :n], eh[:, n:]
    f = act(g, name)[0]
    ef = SLOPE * eg + act_error(g) * np.abs(f)
    return f * u, ef * np.abs(u) + np.abs(f) * eu + ef * eu + 2.0 ** -22 * np.abs(f * u)


def gated_gradient(d, ed, h, name):
    """dh and act(gate) up of exact h, from d and its error, with their errors."""
    n = h.shape[1] // 2
    g, u = h[:, :n], h[:, n:]
    f, s = act(g, name)
    es, ef = act_error(g), act_error(g) * np.abs(f)
    dg, du = d * u * s, d * f
    eg = np.abs(u) * (np.abs(s) * ed + es * (np.abs(d) + ed)) + 2.0 ** -22 * np.abs(dg)
    eu = np.abs(f) * ed + ef * (np.abs(d) + ed) + 2.0 ** -22 * np.abs(du)
    out = f * u
    return np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1), out, ef * np.abs(u) + 2.0 ** -22 * np.abs(out)


def check_bf16(got, want, err, what):
    """A BF16 output within half a step of a value that is off by err, and in the 2-norm."""
    bound = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * err + 2.0 ** -133
    bad = np.argwhere(~(np.abs(got - want) <= bound))
    assert not len(bad), (what, len(bad), bad[:5], got[tuple(bad[0])], want[tuple(bad[0])])
    assert np.linalg.norm(got - want) <= 2.0 ** -8 * np.linalg.norm(want), what


def check_fp8(q, scales, want, err, what):
    """E4M3 bytes and FP32 scales per 1x128 block of a value that is off by err: each scale is
    its block's amax / 448, each byte within half a step (2^-4 of the value, 2^-10 of the scale
    below the smallest normal number)."""
    kb = -(-want.shape[1] // 128)
    assert scales.shape[1] == kb
    # a byte rounds to nearest: rms error 2^-4 / sqrt(3) of a value at most
    v = ref.e4m3(q) * scales.astype(np.float64)[:, np.arange(want.shape[1]) // 128]
    for b in range(kb):
        c = slice(128 * b, 128 * b + 128)
        amax = np.maximum(np.abs(want[:, c]).max(1), 2.0 ** -100)
        off = err[:, c].max(1) + 2.0 ** -22 * amax
        assert (np.abs(scales[:, b].astype(np.float64) * 448 - amax) <= off).all(), (what, b)
        s = scales[:, b:b + 1].astype(np.float64)
        bound = np.maximum(2.0 ** -4 * np.abs(want[:, c]), 2.0 ** -10 * s) + (1 + 2.0 ** -4) * err[:, c] \
            + 2.0 ** -21 * np.abs(want[:, c])
        bad = np.argwhere(~(np.abs(v[:, c] - want[:, c]) <= bound))
        assert not len(bad), (what, b, len(bad), bad[:5])
    assert np.linalg.norm(v - want) <= 2.0 ** -4 / np.sqrt(3) * np.linalg.norm(want) + 2.0 ** -100, what

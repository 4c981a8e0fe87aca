"""The activations' formulas in emulated FP32 against their bounds, and the normal tail's
polynomial against the best one (CPU)."""
from __future__ import annotations

import os
import re

import numpy as np
import pytest
from scipy.special import erfcx

import act_bounds as ab
import ffn_ref as fr

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "block_scaled_precision_bf16tofp4row_amd", "csrc", "activation.h")


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_formulas_within_their_bounds(name):
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        for x in (ab.bf16_numbers().ravel(), ab.arguments(1 << 20, 5)):
            x64 = np.clip(x.astype(np.float64), -1e4, None)       # (both are 0 there, and 1 to the right)
            got, got_slope = ab.emulated(x, name)
            value, slope = fr.act(x64, name)
            slope = np.where(x64 > 1e4, 1, slope)
            assert (np.abs(got - value) <= ab.value_bound(x64, value, name)).all()
            assert (np.abs(got_slope - slope) <= ab.slope_bound(x64, slope, name)).all()


def test_bounds_are_not_loose():
    """Half of them would not do: the emulation has no error of the hardware's functions, but most
    of the rest."""
    for name, part in (("silu", 0.25), ("gelu", 0.25), ("gelu_tanh", 0.25)):
        x = ab.arguments(1 << 20, 6).astype(np.float64)
        got, got_slope = ab.emulated(x, name)
        value, slope = fr.act(x, name)
        assert (np.abs(got - value) > part * ab.value_bound(x, value, name)).any(), name
        assert (np.abs(got_slope - slope) > part * ab.slope_bound(x, slope, name)).any(), name


def test_header_has_these_coefficients():
    with open(HEADER) as f:
        text = f.read()
    gelu = text[text.index("ACT == kActGelu)"):text.index("} else {", text.index("ACT == kActGelu)"))]
    found = [float(v) for v in re.findall(r"q = (?:__builtin_fmaf\(q, t, )?(-?[0-9.]+)f", gelu)]
    assert found == list(ab.TAIL)


def tail(z):
    """P(-z) exp(z^2 / 2) / t with t = 1 / (1 + 0.28 z)."""
    return 0.5 * erfcx(z / np.sqrt(2)) * (1 + 0.28 * z)


def test_tail_polynomial():
    """The committed coefficients against a fit made here for every z >= 0, which is every t in
    (0, 1]: least squares of the relative error over Chebyshev points of t, reweighted by the
    error until it is even."""
    t = 0.5 + 0.5 * np.cos(np.pi * (np.arange(4000) + 0.5) / 4000)
    want = tail((1 / t - 1) / 0.28)
    V = np.vander(t, 9) / want[:, None]
    w, best = np.ones(len(t)), np.inf
    for _ in range(200):
        c = np.linalg.lstsq(V * np.sqrt(w)[:, None], np.sqrt(w), rcond=None)[0]
        e = np.abs(V @ c - 1)
        best = min(best, e.max())
        w *= e / e.max() + 1e-3
        w /= w.mean()
    mine = np.abs(np.polyval(ab.TAIL, t) / want - 1).max()
    # (the coefficients are FP32: of the sum of their magnitudes, 0.7 relative to the smallest value
    # 0.11 of the polynomial's magnitude, half a step each)
    assert best <= 1.8e-7 and mine <= best + 0.7 / 0.11 * 2.0 ** -25, (best, mine)

"""How far the kernels' activations and derivatives (csrc/activation.h) may be off, in units of
u = 2^-24, and their formulas in NumPy's float32.

Roundings: an FP32 operation 1 u of its result; the hardware's 2^x and reciprocal 2 u each.
A relative error of the exponential's argument is E times as large in the exponential, with E
the argument's magnitude:
  silu       E = -x: the product with log2 e 1 u and that constant 0.25 u              1.25 E
  gelu       E = x^2 / 2: another product                                              2.25 E
  gelu_tanh  E = 1.6 |x| + 0.0714 |x|^3: three more products and the constants' 0.5 u
             each at most                                                              6.25 E
Values, relative to themselves: the exponential 2 u, 1 + e 1 u, reciprocal 2 u, product 1 u: 6 u,
for silu and gelu_tanh.  For gelu the fit of the tail with its own evaluation, 5.3e-7 to 6.5e-7
(11 u), t = 1 / (1 + 0.28 z) with 3.3 u, which the tail's polynomial takes by less than two, and
four products: below 24 u.  To the right of zero 1 - P(-x) has no more than half of that, and the
exponential's part vanishes faster than E grows.
Far left, where 1 / (1 + e) is below the smallest normal number or e infinite, a value may come
out as zero: |x| 2^-126 or |x| exp(-88.7), below 2^-121.

Derivatives, which have zeros, absolutely.
  silu       s (1 + x (1 - s)): an error d of s goes in by 1 + x (1 - 2 s), at most 18 in
             magnitude where s is not 1 yet (x < 17), and d is 3 u there: 54 u, and 5 u of the
             products
  gelu_tanh  the same with 1 + (1 - 2 s) x g, g = 1.6 (1 + 0.134 x^2): 29 at x = 4.6, where s
             gets to be 1, with d 3 u: 87 u, 5 u of the exponential's argument and 16 u of
             the products
  gelu       P + x phi(x): half of P's 24 u, phi's error 2.25 E + 4 u times x phi <= 0.242, and the
             sum's rounding, at most 1.13 u: 17 u
Left of -4 the zeros are behind, and a derivative is good relative to itself as well: the value's
error with up to 16 u of products, for gelu 1.3 times (x phi and P differ by that little).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
F = np.float32
#: the coefficients of the tail's polynomial, highest power first, as activation.h has them
TAIL = (0.024720078334212303, -0.09359350055456161, 0.09242866188287735, -0.006449582055211067, 0.07277517020702362,
        0.0836307555437088, 0.10308466851711273, 0.11169980466365814, 0.11170385777950287)
SLOPE = {"silu": 64 * U, "gelu": 32 * U, "gelu_tanh": 128 * U}


def argument(x, name):
    """E of negative arguments, 0 to the right."""
    z = np.maximum(-np.asarray(x, np.float64), 0)
    return {"silu": z, "gelu": z * z / 2, "gelu_tanh": 1.6 * z + 0.0714 * z ** 3}[name]


def value_bound(x, value, name):
    """Absolute, of act(x) = value."""
    a, c = {"silu": (1.25, 6), "gelu": (2.25, 24), "gelu_tanh": (6.25, 6)}[name]
    return (a * argument(x, name) + c) * U * np.abs(value) + 2.0 ** -121


def slope_bound(x, slope, name):
    """Absolute, of act'(x) = slope."""
    a, c = {"silu": (1.25, 22), "gelu": (3, 34), "gelu_tanh": (6.25, 22)}[name]
    tail = (a * argument(x, name) + c) * U * np.abs(slope) + 2.0 ** -118
    return np.where(np.asarray(x) <= -4, np.minimum(tail, SLOPE[name]), SLOPE[name])


def _fma(a, b, c):
    return (a.astype(np.float64) * np.float64(b) + np.float64(c)).astype(F)


def _exp(x):
    return np.exp2((x * F(1.4426950408889634)).astype(np.float64)).astype(F)


def _rcp(x):
    return (1 / x.astype(np.float64)).astype(F)


def emulated(x, name):
    """activation.h's formulas, step by step in FP32, with exact 2^x and reciprocals."""
    x = np.asarray(x, F)
    with np.errstate(over="ignore", under="ignore"):
        if name == "silu":
            s = _rcp(F(1) + _exp(-x))
            return x * s, s * _fma(x, F(1) - s, F(1))
        if name == "gelu":
            t, e = _rcp(_fma(np.abs(x), F(0.28), F(1))), _exp(F(-0.5) * x * x)
            q = np.full_like(x, TAIL[0])
            for c in TAIL[1:]:
                q = _fma(q, t, F(c))
            q = q * (t * e)
            p = np.where(x < 0, q, F(1) - q).astype(F)
            return x * p, _fma(x, F(0.3989422804014327) * e, p)
        c = F(1.5957691216057308)
        y = np.clip(x, F(-30), F(30))
        s = _rcp(F(1) + _exp(-c * y * _fma(F(0.044715) * y, y, F(1))))
        return x * s, s * _fma(y * (F(1) - s), c * _fma(F(0.134145) * y, y, F(1)), F(1))


def bf16_numbers():
    """Every finite BF16 number, as float32 [255, 256]."""
    bits = np.arange(1 << 16, dtype=np.uint32)
    return (bits[(bits & 0x7F80) != 0x7F80] << 16).view(F).reshape(255, 256)


def arguments(n, seed):
    """FP32 arguments: about zero, over the tails, and of every magnitude."""
    rng = np.random.default_rng(seed)
    x = np.concatenate([rng.uniform(-6, 6, n // 2), rng.uniform(-30, 10, n // 4), rng.uniform(-86, 0, n // 8),
                        rng.choice([-1, 1], n // 8) * 2.0 ** rng.uniform(-60, 6, n // 8)])
    return rng.permutation(x).astype(F)

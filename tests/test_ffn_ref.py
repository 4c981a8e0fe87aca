"""The feed-forward references themselves: derivatives against differences, and values against
torch's functions (CPU)."""
import numpy as np
import pytest
import torch

import ffn_ref as fr


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_derivative_is_the_slope(name):
    x = np.linspace(-9, 9, 4001) + 1e-3
    e = 1e-5
    d = (fr.act(x + e, name)[0] - fr.act(x - e, name)[0]) / (2 * e)
    s = fr.act(x, name)[1]
    assert np.abs(d - s).max() < 1e-8
    assert np.abs(s).max() <= fr.SLOPE


def test_values():
    x = torch.linspace(-12, 12, 1001, dtype=torch.float64)
    f = torch.nn.functional
    for name, want in (("relu", f.relu(x)), ("silu", f.silu(x)), ("gelu", f.gelu(x)),
                       ("gelu_tanh", f.gelu(x, approximate="tanh"))):
        np.testing.assert_allclose(fr.act(x.numpy(), name)[0], want.numpy(), rtol=1e-9, atol=1e-14)


def test_gated_gradient_against_differences():
    rng = np.random.default_rng(3)
    h, d = rng.normal(size=(4, 12)), rng.normal(size=(4, 6))
    zero = np.zeros_like(d)
    dh, _, out, _ = fr.gated_gradient(d, zero, h, "gelu")
    assert np.allclose(out, fr.gated_out(h, np.zeros_like(h), "gelu")[0])
    for m, n in ((0, 0), (1, 5), (2, 6), (3, 11)):
        step = np.zeros_like(h)
        step[m, n] = 1e-6
        up, down = (fr.gated_out(h + s, np.zeros_like(h), "gelu")[0] for s in (step, -step))
        assert abs(((up - down) * d).sum() / 2e-6 - dh[m, n]) < 1e-7

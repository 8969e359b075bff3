"""Pins of the activation oracle: torch's definitions, differences, and the error bounds'
agreement with a float32 restatement of the kernels' formulas."""

import numpy as np
import pytest
import torch

from oracle import act as OA

Z = np.concatenate([np.linspace(-12, 12, 4801), [-80.0, -30.0, 30.0, 80.0]])
TORCH = {OA.RELU: torch.relu, OA.SILU: torch.nn.functional.silu,
         OA.GELU: lambda t: torch.nn.functional.gelu(t, approximate="tanh")}


@pytest.mark.parametrize("kind", [OA.RELU, OA.GELU, OA.SILU])
def test_values_and_slopes_are_torchs(kind):
    z = torch.tensor(Z, dtype=torch.float64, requires_grad=True)
    y = TORCH[kind](z)
    y.sum().backward()
    # gelu by tanh cancels at z << 0 in torch's form: 2^-53 |z| absolute
    np.testing.assert_allclose(OA.act(Z, kind), y.detach().numpy(), rtol=1e-13, atol=1e-14)
    np.testing.assert_allclose(OA.slope(Z, kind), z.grad.numpy(), rtol=1e-12, atol=1e-13)


@pytest.mark.parametrize("kind", [OA.NONE, OA.GELU, OA.SILU])
def test_slope_against_differences(kind):
    z, d = np.linspace(-6, 6, 97) + 0.01, 1e-5
    num = (OA.act(z + d, kind) - OA.act(z - d, kind)) / (2 * d)
    assert np.max(np.abs(num - OA.slope(z, kind))) < 1e-8


def test_backward_of_the_gated_form_against_autograd():
    g = torch.Generator().manual_seed(0)
    z, u, dy = (torch.randn(5, 7, generator=g, dtype=torch.float64) for _ in range(3))
    z.requires_grad_(), u.requires_grad_()
    (torch.nn.functional.silu(z) * u).backward(dy)
    dz, du = OA.backward(dy.numpy(), z.detach().numpy(), OA.SILU, u.detach().numpy())
    np.testing.assert_allclose(dz, z.grad.numpy(), rtol=1e-12)
    np.testing.assert_allclose(du, u.grad.numpy(), rtol=1e-12)
    dz, du = OA.backward(dy.numpy(), z.detach().numpy(), OA.RELU)
    assert du is None and np.array_equal(dz, dy.numpy() * (z.detach().numpy() > 0))


@pytest.mark.parametrize("kind", [OA.GELU, OA.SILU])
def test_error_bounds_cover_float32_arithmetic(kind):
    """The kernels' formulas in numpy float32 (exact to its own rounding) stay inside the bounds."""
    z = Z.astype(np.float32)
    one = np.float32(1)
    if kind == OA.GELU:
        s = np.minimum(z * z, np.float32(1e30))
        w = z * (np.float32(1.5957691216057308 * 0.044715) * s + np.float32(1.5957691216057308))
        dw = np.float32(3 * 1.5957691216057308 * 0.044715) * s + np.float32(1.5957691216057308)
    else:
        w, dw = z, one
    t = np.exp(-np.abs(w))
    r = one / (one + t)
    p, q = np.where(w >= 0, r, t * r), np.where(w >= 0, t * r, r)
    assert np.all(np.abs(z * p - OA.act(z, kind)) <= OA.value_error(z, kind) + 2.0 ** -126)
    assert np.all(np.abs(p + z * p * q * dw - OA.slope(z, kind)) <= OA.slope_error(z, kind))

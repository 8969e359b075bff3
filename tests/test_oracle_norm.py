"""Pins of the norm oracle: closed forms, hand-worked rows, and differences."""

import numpy as np
import pytest
import torch

from oracle import fp8_formats as F
from oracle import norm as ON


def test_hand_worked_row():
    # mean(h^2) = (9 + 16) / 2 = 12.5; eps 12.5 makes rstd exactly 1/5.
    y, rstd = ON.rmsnorm([[3.0, -4.0]], [1.0, 2.0], 12.5)
    assert rstd[0] == 0.2
    np.testing.assert_allclose(y, [[0.6, -1.6]], rtol=1e-15)


def test_unit_rows_have_unit_mean_square():
    h = np.random.default_rng(0).normal(size=(5, 33)) * 7
    y, _ = ON.rmsnorm(h, np.ones(33), 1e-300)
    np.testing.assert_allclose(np.mean(y * y, axis=1), 1.0, rtol=1e-12)


@pytest.mark.parametrize("dres", [False, True])
def test_gradient_against_differences(dres):
    rng = np.random.default_rng(1)
    h, gamma, dy = rng.normal(size=(3, 6)), rng.normal(size=6), rng.normal(size=(3, 6))
    extra = rng.normal(size=(3, 6)) if dres else None
    eps = 1e-3

    def loss(h, gamma):
        y = ON.rmsnorm(h, gamma, eps)[0]
        return np.sum(dy * y) + (np.sum(extra * h) if dres else 0.0)

    _, rstd = ON.rmsnorm(h, gamma, eps)
    dx, dgamma = ON.rmsnorm_backward(dy, h, rstd, gamma, extra)
    d = 1e-5
    for i in np.ndindex(h.shape):
        e = np.zeros_like(h)
        e[i] = d
        # Central differences of a smooth function: error O(d^2) plus rounding 1e-16 / d.
        assert abs((loss(h + e, gamma) - loss(h - e, gamma)) / (2 * d) - dx[i]) < 1e-8
    for i in range(6):
        e = np.zeros(6)
        e[i] = d
        assert abs((loss(h, gamma + e) - loss(h, gamma - e)) / (2 * d) - dgamma[i]) < 1e-8


def test_gradient_against_autograd():
    g = torch.Generator().manual_seed(2)
    h = torch.randn(4, 9, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(9, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(4, 9, generator=g, dtype=torch.float64)
    (h * (h.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt() * w).backward(dy)
    _, rstd = ON.rmsnorm(h.detach().numpy(), w.detach().numpy(), 1e-6)
    dx, dgamma = ON.rmsnorm_backward(dy.numpy(), h.detach().numpy(), rstd, w.detach().numpy())
    np.testing.assert_allclose(dx, h.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dgamma, w.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_row_scales_reach_the_largest_code_and_skip_empty_rows():
    y = np.array([[1.0, -3.5], [0.0, 0.0], [np.inf, 1.0]])
    s = ON.row_scales(y, F.E4M3)
    assert s[0] == 128.0 and s[1] == 1.0 and s[2] == 1.0
    assert F.encode(y[:1] * s[0], F.E4M3)[0, 1] == 0xFE  # -448

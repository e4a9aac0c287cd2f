"""Pins of the float64 RMS norm: by hand, against differences, against torch's autograd."""
import numpy as np
import pytest

from oracle import rmsnorm

pytestmark = pytest.mark.cpu


def test_forward_by_hand():
    s = np.array([[3.0, 4.0], [0.0, 0.0]])
    y, r = rmsnorm.forward(s, np.array([2.0, 1.0]), 0.25)
    # mean square 12.5 + 0.25 = 12.75; a zero row takes eps alone
    assert np.allclose(r, [12.75 ** -0.5, 2.0])
    assert np.allclose(y, [[6.0 * 12.75 ** -0.5, 4.0 * 12.75 ** -0.5], [0.0, 0.0]])


def _case(seed, T=3, H=8):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((T, H)), 1.0 + 0.3 * rng.standard_normal(H), rng.standard_normal((T, H)),
            rng.standard_normal((T, H)))


def test_backward_against_differences():
    s, gamma, dy, ds_in = _case(1)
    eps, h = 1e-2, 1e-6

    def loss(s, gamma):
        return np.sum(dy * rmsnorm.forward(s, gamma, eps)[0]) + np.sum(ds_in * s)

    ds, dgamma = rmsnorm.backward(dy, s, gamma, rmsnorm.rstd(s, eps), ds_in)
    for idx in np.ndindex(s.shape):
        e = np.zeros_like(s)
        e[idx] = h
        # central differences: h^2 truncation and 1e-16 / h cancellation, both far below 1e-7
        assert abs((loss(s + e, gamma) - loss(s - e, gamma)) / (2 * h) - ds[idx]) < 1e-7
    for i in range(gamma.size):
        e = np.zeros_like(gamma)
        e[i] = h
        assert abs((loss(s, gamma + e) - loss(s, gamma - e)) / (2 * h) - dgamma[i]) < 1e-7


def test_backward_against_autograd():
    torch = pytest.importorskip("torch")
    s, gamma, dy, ds_in = _case(2, 5, 32)
    st, gt = torch.tensor(s, requires_grad=True), torch.tensor(gamma, requires_grad=True)
    y = st * torch.rsqrt(st.square().mean(1, keepdim=True) + 1e-6) * gt
    ((y * torch.tensor(dy)).sum() + (st * torch.tensor(ds_in)).sum()).backward()
    ds, dgamma = rmsnorm.backward(dy, s, gamma, rmsnorm.rstd(s, 1e-6), ds_in)
    assert np.allclose(ds, st.grad.numpy(), rtol=1e-12, atol=1e-12)
    assert np.allclose(dgamma, gt.grad.numpy(), rtol=1e-12, atol=1e-12)

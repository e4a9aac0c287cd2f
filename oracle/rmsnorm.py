"""Residual addition and RMS norm in float64 (oracle), forward and backward.

TEST INFRASTRUCTURE ONLY -- see the package docstring.

    s = x + r;  rstd = (mean_h s^2 + eps)^(-1/2);  y = s rstd gamma
    n = s rstd;  ds = rstd (dy gamma - n mean_h(dy gamma n)) + ds_in;  dgamma = sum_t dy n

Nothing is rounded here: the caller rounds where the call under test does.
"""

import numpy as np


def rstd(s, eps):
    return 1.0 / np.sqrt(np.mean(np.square(s), axis=1) + eps)


def forward(s, gamma, eps):
    """(y, rstd) of the rows of s."""
    r = rstd(s, eps)
    return s * r[:, None] * gamma, r


def backward(dy, s, gamma, r, ds_in=None):
    """(ds, dgamma) for the forward's s and rstd r."""
    n = s * r[:, None]
    d = dy * gamma
    ds = r[:, None] * (d - n * np.mean(d * n, axis=1, keepdims=True))
    return ds + (0.0 if ds_in is None else ds_in), np.sum(dy * n, axis=0)

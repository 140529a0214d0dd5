"""fp64 reference of the residual RMS norm and its gradient, test
infrastructure only.  y = h / sqrt(mean(h^2) + eps) * w over the last axis; h
is given as it is stored, since the norm reads it so.
"""
from __future__ import annotations

import numpy as np


def forward(h, w, eps):
    return h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * w


def backward(h, w, dy, eps, dh=None):
    """(d, dw): d reaches both x and the residual."""
    rms = np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n = h / rms
    gw = dy * w
    d = (gw - n * (gw * n).mean(-1, keepdims=True)) / rms
    if dh is not None:
        d = d + dh
    return d, (dy * n).sum(0)


def backward_magnitude(h, w, dy, eps, dh=None):
    """The sums of absolute values that d and dw are made of."""
    rms = np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n, gw = np.abs(h) / rms, np.abs(dy * w)
    d = (gw + n * (gw * n).mean(-1, keepdims=True)) / rms
    return d + (0 if dh is None else np.abs(dh)), (np.abs(dy) * n).sum(0)

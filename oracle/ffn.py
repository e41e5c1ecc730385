"""Gated feed-forward block and its gradients (oracle).

Test infrastructure only (see ``oracle/__init__``).

Plain float64 formulas over decoded values; ``w`` holds the gate projection's
rows, then the up projection's.
"""
from __future__ import annotations

import numpy as np

from . import block as B


def forward(x, w):
    """(y, g, u) for x [M, K], w [2F, K]."""
    F = w.shape[0] // 2
    g, u = x @ w[:F].T, x @ w[F:].T
    return B.swiglu(g, u), g, u


def activation_backward(dy, g, u):
    """[dg | du]."""
    return np.concatenate(B.swiglu_backward(dy, g, u), axis=1)


def gradients(dgu, x, w):
    """(dx, dw)."""
    return dgu @ w, dgu.T @ x

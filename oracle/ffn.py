"""Dense gated feed-forward block and its gradients. float64 CPU definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).

For token rows x [T, H], gate, up [I, H] and down [H, I]:

    g = x gate^T, u = x up^T, h = silu(g) u, y = h down^T

and, from dy and given g and u, the gradients of sum(dy y):

    dh = dy down, dg = dh u s (1 + g (1 - s)), du = dh g s     (s = sigmoid(g))
    dx = dg gate + du up, dgate = dg^T x, dup = du^T x, ddown = dy^T h

No rounding here: the tests add those of the kernels.
"""
from __future__ import annotations

import numpy as np


def sigmoid(g):
    t = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, t) / (1.0 + t)


def hidden(g, u):
    return g * sigmoid(g) * u


def forward(x, gate, up, down):
    """(y, g, u)."""
    g, u = x @ gate.T, x @ up.T
    return hidden(g, u) @ down.T, g, u


def backward(x, g, u, dy, gate, up, down):
    """(dx, dgate, dup, ddown)."""
    s, dh = sigmoid(g), dy @ down
    dg, du = dh * u * s * (1.0 + g * sigmoid(-g)), dh * g * s
    return dg @ gate + du @ up, dg.T @ x, du.T @ x, dy.T @ hidden(g, u)

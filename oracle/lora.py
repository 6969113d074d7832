"""Low-rank adapters beside a shared projection, and their gradients. float64
CPU definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).

For token row x_t with adapter a = adapter[t] (an index outside 0 .. n - 1: no
adapter, and nothing is added):

    y_t  = base_t + s_a B_a (A_a x_t)
    g_t  = s_a B_a^T dy_t,  h_t = s_a A_a x_t
    dx_t = dx_base_t + A_a^T g_t
    dA_a = sum_t g_t x_t^T,  dB_a = sum_t dy_t h_t^T

No rounding here: the tests add the output's.
"""
from __future__ import annotations

import numpy as np


def apply(x, adapter, A, B, scale, base):
    """y [T, N] in float64 from x [T, K], A [n, R, K], B [n, N, R], scale [n]."""
    y = np.array(base, np.float64)
    for t, a in enumerate(adapter):
        if 0 <= a < len(A):
            y[t] += np.float64(scale[a]) * (B[a] @ (A[a] @ x[t]))
    return y


def backward(x, dy, adapter, A, B, scale, dx_base):
    """(dx, dA, dB) in float64."""
    dx, dA, dB = np.array(dx_base, np.float64), np.zeros_like(A, np.float64), np.zeros_like(B, np.float64)
    for t, a in enumerate(adapter):
        if 0 <= a < len(A):
            g = np.float64(scale[a]) * (B[a].T @ dy[t])
            h = np.float64(scale[a]) * (A[a] @ x[t])
            dx[t] += A[a].T @ g
            dA[a] += np.outer(g, x[t])
            dB[a] += np.outer(dy[t], h)
    return dx, dA, dB

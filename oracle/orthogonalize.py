"""Newton-Schulz steps on a matrix. float64 CPU definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).

With M = U diag(sigma) V^T and s = sigma / (|M| + eps), each step (a, b, c) takes
s to a s + b s^3 + c s^5; the result is scale U diag(s) V^T. Written here through
the singular value decomposition, not through products of matrices.
"""
from __future__ import annotations

import numpy as np


def orthogonalize(m, coeffs, eps, scale=1.0):
    u, sigma, vt = np.linalg.svd(np.asarray(m, np.float64), full_matrices=False)
    s = sigma / (np.sqrt((sigma * sigma).sum()) + eps)
    for a, b, c in coeffs:
        s = s * (a + b * s ** 2 + c * s ** 4)
    return scale * (u * s) @ vt

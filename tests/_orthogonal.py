"""How far an update may be from the exact one, from the arithmetic of its steps and the matrix's own singular values.

A step takes S from X's f16 values and rounds it, P = b S + c S S and rounds it, and P X from X's f16 values, so that with
roundings of at most r relative to a value, a singular value s and p = b s^2 + c s^4, it adds
    dS = (2 r_X + r_S) s^2,   dP = |b + 2 c s^2| dS + r_P |p|,   s (dP + r_X |p|)
and what came before is carried through it by the polynomial's slope a + 3 b s^2 + 5 c s^4. (An error that turns singular
vectors instead is carried as it is, and is no larger.) Up to 32 rows X, S and P are two f16 values each, r = 2^-21: all
errors are taken at their largest and none to cancel, the slope at least one in relative terms, and S's sum over the long
side, k values in steps of 16, loses 2^-23 a step. Above, X and S are one
(r = 2^-11) and P is from 65 rows on: independent roundings, of which many meet in a result, each with a root mean square of
r / sqrt(3), add up in squares.
"""
import numpy as np


def steps_error(m, steps, eps):
    """The norm of the steps' error relative to the result's."""
    sigma = np.linalg.svd(np.asarray(m, np.float64), compute_uv=False)
    s = sigma / (np.sqrt((sigma * sigma).sum()) + eps)
    rows, k = min(m.shape), max(m.shape)
    r_x, r_p = (2.0 ** -21 if rows <= most else 2.0 ** -11 / np.sqrt(3) for most in (32, 64))
    e = np.zeros_like(s)
    for a, b, c in steps:
        q = s * s
        p, via_s, slope = b * q + c * q * q, np.abs(b + 2 * c * q) * q, np.abs(a + 3 * b * q + 5 * c * q * q)
        if rows <= 32:
            e = np.maximum(slope, np.abs(a + p)) * e + s * (via_s * (3 * r_x + k / 16 * 2.0 ** -23) + (r_p + r_x) * np.abs(p))
        else:
            e = np.sqrt((slope * e) ** 2 + s * s * (via_s ** 2 * 3 * r_x ** 2 + (r_p ** 2 + r_x ** 2) * p * p))
        s = s * (a + p)
    return np.sqrt((e * e).sum() / (s * s).sum())


def rounded(ref):
    """The result's own rounding to bf16, relative to its norm (of values as they are)."""
    import torch
    r = torch.from_numpy(ref).to(torch.bfloat16).double().numpy()
    return np.linalg.norm(r - ref) / np.linalg.norm(ref)

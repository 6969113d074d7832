"""Inputs and error bounds of the dense block's and the orthogonalised update's tests.

Bounds are derived from the arithmetic, element by element, before any run, as in _finetune: u = 2^-23 of the sum of
absolute values for each term of an FP32 sum, 2^-8 of a value for its rounding to bf16. The sigmoid's hardware
exponential is off by 2 + 1.2 |g| steps of 2^-23 and its quotient by two: with |g| up to 24, FN = 2^-18 of the value.
silu's slope is below 1.1.
    |dg| = (H + 2) u |x||gate|                        (and du)
    |dh| = 1.1 |dg||u| + |silu(g)||du| + (2^-8 + FN) |h|
    |dy| = 2^-8 |y| + |dh||down| + (I + 2) u |h||down|
Gradients, from given g and u, with k1 = s (1 + g (1 - s)) whose two terms may cancel:
    |d(dy down)| = (H + 2) u |dy||down| = e
    |ddg| = |u k1| e + |dh||u| s (1 + |g| (1 - s)) FN + 2^-8 |dg|
    |ddu| = |g s| e + |du| FN + 2^-8 |du|
and through the last products, whose sums run over 2 I (dx) or T terms. Everything is scaled by 1 + 2^-6 for the
products of these errors.
"""
import numpy as np
import torch

from _finetune import HALF_BF16, SLACK, SUM, TINY, bf16, f64
from oracle import ffn as offn

FN = 2.0 ** -18


class Block:
    """A dense block's weights, tokens and gradients drawn on the CPU from one seed."""

    def __init__(self, T, H, I, seed, sigma=1.0):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.T, self.H, self.I = T, H, I
        self.gate, self.up = bf16(rnd(I, H) * sigma * H ** -0.5), bf16(rnd(I, H) * H ** -0.5)
        self.down = bf16(rnd(H, I) * I ** -0.5)
        self.x, self.dy = bf16(rnd(T, H)), bf16(rnd(T, H))
        _, gg, uu = offn.forward(*(f64(v) for v in (self.x, self.gate, self.up, self.down)))
        self.g, self.u = (bf16(torch.from_numpy(v)) for v in (gg, uu))

    def to(self, dev):
        for k in ("gate", "up", "down", "x", "dy", "g", "u"):
            setattr(self, "d_" + k, getattr(self, k).to(dev))
        return self

    def expect_forward(self):
        """((y, g, u), (bounds))."""
        x, wg, wu, wd = (f64(v) for v in (self.x, self.gate, self.up, self.down))
        y, g, u = offn.forward(x, wg, wu, wd)
        h = offn.hidden(g, u)
        eg, eu = ((self.H + 2) * SUM * (np.abs(x) @ np.abs(w).T) for w in (wg, wu))
        eh = 1.1 * eg * np.abs(u) + np.abs(g * offn.sigmoid(g)) * eu + (HALF_BF16 + FN) * np.abs(h)
        ey = HALF_BF16 * np.abs(y) + (eh + (self.I + 2) * SUM * np.abs(h)) @ np.abs(wd).T
        return (y, g, u), tuple(v * SLACK + TINY for v in (ey, HALF_BF16 * np.abs(g) + eg, HALF_BF16 * np.abs(u) + eu))

    def expect_backward(self):
        """((dx, dgate, dup, ddown), (bounds))."""
        x, g, u, dy, wg, wu, wd = (f64(v) for v in (self.x, self.g, self.u, self.dy, self.gate, self.up, self.down))
        refs = offn.backward(x, g, u, dy, wg, wu, wd)
        s, q = offn.sigmoid(g), offn.sigmoid(-g)
        dh, e = np.abs(dy @ wd), (self.H + 2) * SUM * (np.abs(dy) @ np.abs(wd))
        k1, act, h = np.abs(u * s * (1 + g * q)), np.abs(g * s), np.abs(g * s * u)
        dg, du = dh * k1, dh * act
        eg = k1 * e + dh * np.abs(u) * s * (1 + np.abs(g) * q) * FN + HALF_BF16 * dg
        eu = act * e + (FN + HALF_BF16) * du
        eh = (FN + HALF_BF16) * h
        c = (2 * self.I + 2) * SUM
        ex = (eg + c * dg) @ np.abs(wg) + (eu + c * du) @ np.abs(wu)
        c = (self.T + 2) * SUM
        ew = ((eg + c * dg).T @ np.abs(x), (eu + c * du).T @ np.abs(x), np.abs(dy).T @ (eh + c * h))
        return refs, tuple((HALF_BF16 * np.abs(r) + t) * SLACK + TINY for r, t in zip(refs, (ex, *ew)))


def near(got, ref, limit, label):
    """The error's norm against the reference's."""
    got = f64(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), label
    err, size = np.linalg.norm(got - ref), np.linalg.norm(ref)
    assert err <= limit * size, f"{label}: {err / size if size else err:.2e} above {limit:.2e}"


STEPS = ((3.4445, -4.7750, 2.0315),) * 5


def momentum(n, rows, cols, seed, kind="fading"):
    """Matrices as updates are: a few strong directions over noise, noise alone, or one direction far above the rest."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    r = min(16, rows, cols)
    if kind == "noise":
        return rnd(n, rows, cols)
    if kind == "spike":
        return 1000 * rnd(n, rows, 1) @ rnd(n, 1, cols) + rnd(n, rows, cols)
    return 1e-3 * ((rnd(n, rows, r) * torch.exp(-torch.arange(r) / 3.0)) @ rnd(n, r, cols) + 0.2 * rnd(n, rows, cols))

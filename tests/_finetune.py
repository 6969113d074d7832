"""Inputs and error bounds of the fine-tuning operators' tests.

Bounds are derived from the arithmetic, element by element, before any run. With
u = 2^-24 (FP32), |.| sums taken in float64, and every FP32 sum of n products
allowed n * 2^-23 of the sum of their absolute values (tensor-core sums may
truncate, which is twice a rounding):
  h = s A x              |dh| <= (K + 2) 2^-23 |s| |A||x| + 2^-16 |h|   (hi + lo bf16 halves: 2^-8 * 2^-8)
  y = bf16(base + B h)   |dy| <= 2^-8 |y| + |B| |dh| + (2 R + 2) 2^-23 (|base| + |B||h|)
and the same with the roles of A and B exchanged for g and dx; for the weights'
gradients the sums run over the adapter's tokens. Everything is scaled by 1 + 2^-6
for the products of these errors.
"""
import numpy as np
import torch

from oracle import lora as olora

HALF_BF16 = 2.0 ** -8
SUM = 2.0 ** -23
SLACK = 1 + 2.0 ** -6
TINY = 2.0 ** -126


def bf16(t):
    return t.to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


class Pool:
    """Adapters, tokens and gradients drawn on the CPU from one seed."""

    def __init__(self, T, K, N, R, n, seed, adapter=None):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.T, self.K, self.N, self.R, self.n = T, K, N, R, n
        self.A, self.B = bf16(rnd(n, R, K) * K ** -0.5), bf16(rnd(n, N, R) * R ** -0.5)
        self.scale = torch.rand(n, generator=g) + 0.25
        self.x, self.y, self.dy, self.dx = (bf16(rnd(T, d)) for d in (K, N, N, K))
        if adapter is None:
            adapter = torch.randint(-1, n, (T,), generator=g)
        self.adapter = torch.as_tensor(adapter, dtype=torch.int32)

    def live(self):
        a = self.adapter.numpy()
        return (a >= 0) & (a < self.n)

    def f64(self):
        return tuple(f64(v) for v in (self.x, self.A, self.B, self.scale))

    def _low(self, v, W, s):
        """|dh| and |h| of h = s W v, W [R, D]."""
        h = np.abs(s * (v @ W.T))
        return (W.shape[1] + 2) * SUM * abs(s) * (np.abs(v) @ np.abs(W).T) + 2.0 ** -16 * h, h

    def expect_apply(self, base):
        """(y, bound) in float64 for a float64 base."""
        x, A, B, s = self.f64()
        a = self.adapter.numpy()
        y = olora.apply(x, a, A, B, s, base)
        tol = HALF_BF16 * np.abs(y)
        for i in range(self.n):
            t = np.nonzero(a == i)[0]
            dh, h = self._low(x[t], A[i], s[i])
            tol[t] += dh @ np.abs(B[i]).T + (2 * self.R + 2) * SUM * (np.abs(base[t]) + h @ np.abs(B[i]).T)
        return y, tol * SLACK + TINY

    def expect_backward(self):
        """((dx, dA, dB), (bounds))."""
        x, A, B, s = self.f64()
        dy, dx0, a = f64(self.dy), f64(self.dx), self.adapter.numpy()
        dx, dA, dB = olora.backward(x, dy, a, A, B, s, dx0)
        tx, tA, tB = (HALF_BF16 * np.abs(v) for v in (dx, dA, dB))
        for i in range(self.n):
            t = np.nonzero(a == i)[0]
            dh, h = self._low(x[t], A[i], s[i])
            dg, g = self._low(dy[t], B[i].T, s[i])
            tx[t] += dg @ np.abs(A[i]) + (2 * self.R + 2) * SUM * (np.abs(dx0[t]) + g @ np.abs(A[i]))
            c = (2 * len(t) + 2) * SUM
            tA[i] += (dg + c * g).T @ np.abs(x[t])
            tB[i] += np.abs(dy[t]).T @ (dh + c * h)
        return (dx, dA, dB), tuple(v * SLACK + TINY for v in (tx, tA, tB))

    def to(self, dev):
        for k in ("A", "B", "scale", "x", "y", "dy", "dx", "adapter"):
            setattr(self, "d_" + k, getattr(self, k).to(dev))
        return self


def check(got, ref, tol, label):
    got = f64(got)
    assert got.shape == ref.shape, label
    assert np.all(np.isfinite(got)), label
    err = np.abs(got - ref)
    worst = float((err / tol).max()) if err.size else 0.0
    assert np.all(err <= tol), f"{label}: {int((err > tol).sum())} of {err.size} beyond the bound, worst {worst:.3f}x"


def router(T, E, k, seed, bounds=None, sigma=1.0, pad=(), drop=()):
    """Logits, picks and sequence starts on the CPU: picks are the k largest logits."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * sigma + torch.randn(E, generator=g) * 0.5
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32) if T else torch.zeros(0, k, dtype=torch.int32)
    for t in pad:
        idx[t] = -1
    for t, j in drop:
        idx[t, j] = E + 3
    dw = torch.randn(T, k, generator=g)
    start = None if bounds is None else torch.tensor(bounds, dtype=torch.int32)
    return z, idx, start, dw

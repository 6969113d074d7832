"""Balance loss of the router, per-expert counts, and the logits' gradient.
float64 CPU definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).

    s_te = sigmoid(z_te),  p_t = softmax(log s_t) = s_t / sum s_t
    f_be = E c_be / (k T_b)
    loss = alpha / n_seq  sum_b 1/T_b  sum_{t in b} sum_e f_be p_te
    dz_tj = dloss alpha / (n_seq T_b) p_tj (f_bj - f_b . p_t) (1 - s_tj)
            + sum over picks i of dw_ti d w_ti / d z_tj
    w_ti = routed_scale s_i / sum_picks s   (renormalised; else routed_scale s_i)

Sequence b is the tokens start[b] .. start[b + 1] - 1. A token whose first pick
is negative is padding; another pick outside 0 .. E - 1 is dropped. Rows of
tokens in no sequence are NaN in the gradient returned here (not computed).
"""
from __future__ import annotations

import numpy as np


def log_sigmoid(z):
    return np.where(z >= 0, -np.log1p(np.exp(-np.abs(z))), np.where(z > -np.inf, z, -np.inf) - np.log1p(np.exp(-np.abs(z))))


def shares(z):
    """softmax(log sigmoid(z)); zeros for a row that is all -inf."""
    ls = log_sigmoid(np.asarray(z, np.float64))
    m = ls.max()
    if m == -np.inf:
        return np.zeros_like(ls)
    e = np.exp(ls - m)
    return e / e.sum()


def one_minus_sigmoid(z):
    return np.exp(log_sigmoid(-np.asarray(z, np.float64)))


def picks(row, E):
    return [int(e) for e in row if 0 <= e < E]


def counts(idx, start, E):
    """(seq_counts [n, E], seq_tokens [n])."""
    n = len(start) - 1
    c, tok = np.zeros((n, E), np.int64), np.zeros(n, np.int64)
    for b in range(n):
        for t in range(start[b], start[b + 1]):
            if idx[t][0] < 0:
                continue
            tok[b] += 1
            for e in picks(idx[t], E):
                c[b, e] += 1
    return c, tok


def loss(z, idx, start, k, alpha):
    E = z.shape[1]
    c, tok = counts(idx, start, E)
    total = 0.0
    for b in range(len(start) - 1):
        if tok[b] == 0:
            continue
        f = E * c[b] / (k * tok[b])
        total += sum(float(f @ shares(z[t])) for t in range(start[b], start[b + 1]) if idx[t][0] >= 0) / tok[b]
    return alpha / (len(start) - 1) * total


def backward(z, idx, start, k, alpha, dloss=1.0, dw=None, renormalize=True, routed_scale=1.0):
    T, E = z.shape
    c, tok = counts(idx, start, E)
    n = len(start) - 1
    dz = np.full((T, E), np.nan)
    for b in range(n):
        for t in range(start[b], start[b + 1]):
            dz[t] = 0.0
            if idx[t][0] < 0:
                continue
            f, p, q = E * c[b] / (k * tok[b]), shares(z[t]), one_minus_sigmoid(z[t])
            dz[t] = dloss * alpha / (n * tok[b]) * p * (f - f @ p) * q
            if dw is None:
                continue
            at = [j for j in range(len(idx[t])) if 0 <= idx[t][j] < E]
            e = np.array([idx[t][j] for j in at])
            g = np.array([dw[t][j] for j in at], np.float64)
            if renormalize:
                w = shares(z[t][e])
                d = routed_scale * w * (g - g @ w) * q[e]
            else:
                d = routed_scale * np.exp(log_sigmoid(z[t][e])) * g * q[e]
            np.add.at(dz[t], e, d)
    return dz

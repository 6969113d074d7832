"""Balance loss, per-expert counts and the router's gradient (through the C ABI)
against the float64 definition.

Bounds, derived before any run. u = 2^-24. exp(-z) from the hardware exponential
is within 2 u + |z| 2^-22 of its value (the argument's product is rounded once),
the quotient within 2 ulp, so s and 1 - s are within r = (|z| 4 + 16) u of theirs,
|z| the row's largest; a sum of E positive terms adds (E / 32 + 5) u.
f - 1 is a whole number divided once.
  loss: relative (r + (E / 16 + 16) u), FP64 over the tokens
  dz:   each of p, q, (f - 1) - F is within that of its own parts:
        |c p q| (|f - 1| + sum |f - 1| p) (4 r + (E / 8 + 32) u)
        and the routing weights' part likewise with |dw| + sum |dw| w.
"""
import numpy as np
import pytest
import torch

from oracle import balance as ob
from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _finetune import f64, router

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def cfg_of(E, k, **kw):
    return fb.make_config(hidden=256, num_experts=E, top_k=k, inter=64, **kw)


def forward(z, idx, start, k, alpha, stream=None):
    T, E = z.shape
    n = 1 if start is None else len(start) - 1
    cfg = cfg_of(E, k)
    new = lambda *s: torch.full(s, -7, dtype=torch.int32, device=DEV)  # noqa: E731
    loss = torch.full((1,), float("nan"), device=DEV)
    counts, sc, st = new(E), new(n, E), new(n)
    ws = torch.full((fb.flint_moe_balance_workspace_bytes(cfg, max(T, 1), n),), 0xFF, dtype=torch.uint8, device=DEV)
    fb.flint_moe_balance(cfg, z.to(DEV), idx.to(DEV), T, None if start is None else start.to(DEV), n, alpha, loss, counts,
                         sc, st, ws, stream=stream)
    torch.cuda.synchronize()
    return loss, counts, sc, st


def gradient(z, idx, start, k, alpha, sc, st, dloss=None, dw=None, **kw):
    T, E = z.shape
    dz = torch.full((T, E), float("nan"), device=DEV)
    fb.flint_moe_balance_backward(cfg_of(E, k, **kw), z.to(DEV), idx.to(DEV), T, None if start is None else start.to(DEV),
                                  1 if start is None else len(start) - 1, alpha, sc, st,
                                  None if dloss is None else torch.tensor([dloss], device=DEV),
                                  None if dw is None else dw.to(DEV), dz)
    torch.cuda.synchronize()
    return dz


def starts(start, T):
    return [0, T] if start is None else start.tolist()


def check_all(z, idx, start, dw, k, alpha=0.5, **kw):
    T, E = z.shape
    zz, ii, at = f64(z), idx.numpy(), starts(start, T)
    loss, counts, sc, st = forward(z, idx, start, k, alpha)
    c0, t0 = ob.counts(ii, at, E)
    assert np.array_equal(sc.cpu().numpy(), c0) and np.array_equal(st.cpu().numpy(), t0)
    assert np.array_equal(counts.cpu().numpy(), c0.sum(0))
    fin = np.where(np.isfinite(zz) & (np.abs(zz) < 1e30), np.abs(zz), 0.0)
    zmax = float(fin.max()) if fin.size else 0.0
    r = (4 * zmax + 16) * U
    ref = ob.loss(zz, ii, at, k, alpha)
    # the relative bound is of 1 + F, whose F part alone is inexact before the FP32 rounding of the loss
    assert abs(float(loss) - ref) <= (r + (E / 16 + 16) * U) * (abs(ref) + alpha), (float(loss), ref)
    for g in (None, dw):
        dz = f64(gradient(z, idx, start, k, alpha, sc, st, 1.5, g, **kw))
        want = ob.backward(zz, ii, at, k, alpha, 1.5, None if g is None else f64(g), **kw)
        assert np.array_equal(np.isnan(dz), np.isnan(want))
        for b in range(len(at) - 1):
            for t in range(at[b], at[b + 1]):
                tol = np.full(E, 1e-37)
                if ii[t][0] >= 0:
                    f1 = E * c0[b] / (k * t0[b]) - 1
                    p, q = ob.shares(zz[t]), ob.one_minus_sigmoid(zz[t])
                    rel = 4 * r + (E / 8 + 32) * U
                    tol += abs(1.5 * alpha / ((len(at) - 1) * t0[b])) * p * q * (np.abs(f1) + np.abs(f1) @ p) * rel
                    if g is not None:
                        e = [int(v) for v in ii[t] if 0 <= v < E]
                        gw = np.abs([f64(g)[t][j] for j in range(k) if 0 <= ii[t][j] < E])
                        w = ob.shares(zz[t][e]) if kw.get("renormalize", True) else np.exp(ob.log_sigmoid(zz[t][e]))
                        np.add.at(tol, e, abs(kw.get("routed_scale", 1.0)) * w * (gw + gw @ w) * q[e] * rel)
                    tol += 2 * U * np.abs(want[t])
                err = np.abs(dz[t] - want[t])
                assert np.all(err <= tol), (t, float((err / tol).max()))
    return loss, sc, st


@pytest.mark.parametrize("T,E,k,bounds", [(1, 1, 1, None), (1, 256, 6, None), (2, 3, 2, [0, 1, 2]), (31, 16, 2, None),
                                          (300, 16, 2, [0, 0, 100, 100, 300]), (70, 130, 5, [0, 33, 70]),
                                          (65, 512, 16, [3, 40, 40, 60]), (200, 37, 3, [0, 1, 199, 200]),
                                          (520, 64, 4, None), (90, 511, 7, [0, 90])])
def test_loss_counts_and_gradient(T, E, k, bounds):
    z, idx, start, dw = router(T, E, k, T + E, bounds, pad=[T // 2] if T > 2 else [], drop=[(0, k - 1)] if k > 1 and T > 30 else [])
    check_all(z, idx, start, dw, k)


def test_renormalisation_and_scale():
    z, idx, start, dw = router(50, 64, 6, 3, [0, 20, 50])
    check_all(z, idx, start, dw, 6, renormalize=False, routed_scale=2.5)
    check_all(z, idx, start, dw, 6, renormalize=True, routed_scale=0.5)


def test_extreme_logits():
    """Experts masked by -inf and by the type's lowest value, rows where every score underflows FP32, saturated
    scores, a row of only -inf."""
    E, k = 32, 4
    z, idx, start, dw = router(40, E, k, 5, [0, 40])
    z[1, 5:20] = -float("inf")
    z[2, 5:20] = torch.finfo(torch.float32).min
    z[3] = -200.0 + 3 * z[3]
    z[4] = torch.finfo(torch.float32).min
    z[5] = 60.0 + z[5]
    z[6] = -float("inf")
    z[7, 3] = float("inf")
    z[8] = -85.0 + z[8]
    z[9] = -100.0
    z[9, 7] = 4.0
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
    check_all(z, idx, start, dw, k)


def test_padding_rows_may_hold_anything():
    z, idx, start, dw = router(64, 48, 3, 7, [0, 30, 64], pad=[0, 17, 63])
    a = check_all(z, idx, start, dw, 3)
    z2 = z.clone()
    z2[[0, 17, 63]] = float("nan")
    idx2 = idx.clone()
    idx2[0] = torch.tensor([-1, 5, 900])
    dw2 = dw.clone()
    dw2[[0, 17, 63]] = float("nan")
    b = forward(z2, idx2, start, 3, 0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[2])
    dz = gradient(z2, idx2, start, 3, 0.5, b[2], b[3], None, dw2)
    assert torch.equal(dz, gradient(z, idx, start, 3, 0.5, a[1], a[2], None, dw)) and not dz[[0, 17, 63]].any()


@pytest.mark.parametrize("T,E", [(40, 32), (1200, 130), (1200, 512)])
def test_a_nan_logit_shows(T, E):
    """A NaN in the row of a token that counts: the loss and that row's gradient are NaN, nothing else changes."""
    k = 3
    z, idx, start, dw = router(T, E, k, T + 1, [0, T // 2, T])
    _, _, sc, st = forward(z, idx, start, k, 0.5)
    want = [gradient(z, idx, start, k, 0.5, sc, st, None, g) for g in (None, dw)]
    bad = [5, T // 2 + 2]
    z[bad[0], E - 1] = float("nan")
    z[bad[1], int(idx[bad[1], 0])] = float("nan")
    loss, counts, sc2, st2 = forward(z, idx, start, k, 0.5)
    assert torch.isnan(loss).all() and torch.equal(sc2, sc) and torch.equal(st2, st)
    rest = [t for t in range(T) if t not in bad]
    for g, w in zip((None, dw), want):
        dz = gradient(z, idx, start, k, 0.5, sc, st, None, g)
        assert torch.isnan(dz[bad]).all() and torch.equal(dz[rest], w[rest])


@pytest.mark.parametrize("T,k", [(50, 1), (400, 4), (300, 12)])
def test_a_single_pick_has_no_weight_gradient(T, k):
    """The weight of a token's only pick that counts is one: its gradient adds exactly nothing."""
    E = 64
    z, idx, start, dw = router(T, E, k, 30 + T, [0, T // 3, T])
    idx[:, : k - 1] = E + 3
    _, _, sc, st = forward(z, idx, start, k, 0.5)
    assert torch.equal(gradient(z, idx, start, k, 0.5, sc, st, None, 1e3 * dw), gradient(z, idx, start, k, 0.5, sc, st))


def test_an_expert_picked_twice_counts_twice():
    z, idx, start, dw = router(20, 16, 4, 8)
    idx[3] = torch.tensor([2, 2, 2, 9])
    idx[4] = torch.tensor([7, 1, 7, 1])
    check_all(z, idx, start, dw, 4)


@pytest.mark.parametrize("T,E", [(3000, 256), (9001, 24)])
def test_many_short_sequences_and_determinism(T, E):
    g = torch.Generator().manual_seed(T)
    cuts = torch.unique(torch.randint(0, T, (T // 6,), generator=g)).tolist()
    bounds = [0] + cuts + cuts[-1:] + [T - 5]
    z, idx, start, dw = router(T, E, 2, 9, sorted(bounds))
    loss, counts, sc, st = forward(z, idx, start, 2, 1e-2)
    c0, t0 = ob.counts(idx.numpy(), start.tolist(), E)
    assert np.array_equal(sc.cpu().numpy(), c0) and np.array_equal(st.cpu().numpy(), t0)
    ref = ob.loss(f64(z), idx.numpy(), start.tolist(), 2, 1e-2)
    assert abs(float(loss) - ref) <= 1e-5 * ref  # (4 |z| + 16 + E / 16 + 16) u is below 2^-17
    assert torch.equal(forward(z, idx, start, 2, 1e-2)[0], loss)
    dz = gradient(z, idx, start, 2, 1e-2, sc, st, None, dw)
    again = gradient(z, idx, start, 2, 1e-2, sc, st, None, dw)
    end = int(start[-1])
    assert torch.equal(dz[:end], again[:end]) and torch.isfinite(dz[:end]).all() and torch.isnan(dz[end:]).all()


def test_zero_tokens():
    z, idx, _, _ = router(0, 16, 2, 1)
    loss, counts, sc, st = forward(z, idx, None, 2, 1.0)
    assert float(loss) == 0.0 and not counts.any() and not sc.any() and not st.any()


def test_gradient_against_differences():
    z, idx, start, dw = router(60, 40, 4, 11, [0, 22, 60])
    _, _, sc, st = forward(z, idx, start, 4, 0.7)
    dz = f64(gradient(z, idx, start, 4, 0.7, sc, st))
    v = np.random.default_rng(0).standard_normal(dz.shape)
    L = lambda e: ob.loss(f64(z) + e * v, idx.numpy(), start.tolist(), 4, 0.7)  # noqa: E731
    num = (L(1e-4) - L(-1e-4)) / 2e-4
    # bound: the gradient's relative error of its parts (below 2^-16 of sum |dz v| here, with f - 1 of order one),
    # the differences' e^2 times a third derivative of order one, and their rounding 2^-52 / e
    assert abs(num - float((dz * v).sum())) <= 2.0 ** -16 * float(np.abs(dz * v).sum()) + 1e-8 + 1e-11


def test_streams_and_graphs():
    z, idx, start, dw = router(500, 128, 6, 12, [0, 100, 480])
    z, idx, start, dw = (v.to(DEV) for v in (z, idx, start, dw))
    cfg = cfg_of(128, 6)
    loss = torch.zeros(1, device=DEV)
    counts, sc, st = (torch.zeros(s, dtype=torch.int32, device=DEV) for s in ((128,), (2, 128), (2,)))
    dz = torch.zeros_like(z)
    ws = torch.empty(fb.flint_moe_balance_workspace_bytes(cfg, 500, 2), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        fb.flint_moe_balance(cfg, z, idx, 500, start, 2, 0.3, loss, counts, sc, st, ws)
        fb.flint_moe_balance_backward(cfg, z, idx, 500, start, 2, 0.3, sc, st, None, dw, dz)
    for seed in (13, 14):
        z2, idx2, _, dw2 = router(500, 128, 6, seed)
        z.copy_(z2), idx.copy_(idx2), dw.copy_(dw2)
        g.replay()
        torch.cuda.synchronize()
        want = forward(z2, idx2, start.cpu(), 6, 0.3)
        assert torch.equal(loss, want[0]) and torch.equal(counts, want[1]) and torch.equal(sc, want[2])
        assert torch.equal(dz[:480], gradient(z2, idx2, start.cpu(), 6, 0.3, want[2], want[3], None, dw2)[:480])
        assert not dz[480:].any()  # tokens behind the last sequence: as they were

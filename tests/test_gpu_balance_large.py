"""The balance loss, its counts and the router's gradient at sizes where a warp works through many rows, on ragged
sequences that need not start at the first token, against the float64 definition computed on the GPU.

Bounds, derived before any run, as in test_gpu_balance.py (u = 2^-24, r = (4 |z| + 16) u for s and 1 - s, a sum of E
positive terms (E / 32 + 5) u): dz as there. The loss adds up to 16 tokens' shares in FP32, those sums in FP32 again
(a warp has at most T / 1000 of them here) and E of them times f - 1: relative to sum |f - 1| p of the tokens
2 r + (E / 8 + 64 + T / 1000) u, and one rounding at the end.
"""
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from test_gpu_balance import U, forward, gradient

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()
    yield
    torch.cuda.empty_cache()


def check_large(z, idx, start, dw, k, alpha=0.5, dloss=1.5, renormalize=True, routed_scale=1.0):
    """Counts, loss and both gradients of finite logits (all on the CPU) against float64."""
    T, E = z.shape
    loss, counts, sc, st = forward(z, idx, start, k, alpha)
    at, n = start.to(DEV).long(), len(start) - 1
    zd, ix, t = z.to(DEV).double(), idx.to(DEV).long(), torch.arange(T, device=DEV)
    seq = torch.searchsorted(at, t, right=True) - 1
    inside = (seq >= 0) & (seq < n)
    seq = torch.where(inside, seq, 0)
    live = inside & (ix[:, 0] >= 0)
    ok = live[:, None] & (ix >= 0) & (ix < E)
    c = torch.bincount((seq[:, None] * E + ix)[ok], minlength=n * E).view(n, E)
    tokens = torch.bincount(seq[live], minlength=n)
    assert torch.equal(sc.long(), c) and torch.equal(st.long(), tokens) and torch.equal(counts.long(), c.sum(0))

    r = (4 * float(z.abs().max()) + 16) * U
    f1 = ((E * c - k * tokens[:, None]).double() / (k * tokens.clamp(min=1))[:, None])[seq]
    p = torch.softmax(torch.nn.functional.logsigmoid(zd), dim=1)
    q = torch.sigmoid(-zd)
    F, G = (f1 * p).sum(1), (f1.abs() * p).sum(1)
    each = torch.where(live, alpha / n / tokens[seq].clamp(min=1), 0.0)
    ref = float((each * (1 + F)).sum())
    tol = float((each * G).sum()) * (2 * r + (E / 8 + 64 + T / 1000) * U) + U * abs(ref)
    assert abs(float(loss) - ref) <= tol, (float(loss), ref, tol)

    rel = 4 * r + (E / 8 + 32) * U
    want = dloss * each[:, None] * p * (f1 - F[:, None]) * q
    bound = abs(dloss) * each[:, None] * p * q * (f1.abs() + G[:, None]) * rel
    for g in (None, dw):
        if g is not None:
            g = torch.where(ok, g.to(DEV).double(), 0.0)
            e = ix.clamp(0, E - 1)
            pick = torch.where(ok, torch.nn.functional.logsigmoid(torch.gather(zd, 1, e)), -float("inf"))
            w = torch.nan_to_num(torch.softmax(pick, dim=1), nan=0.0) if renormalize else torch.exp(pick)
            shift, size = (((g * w).sum(1, keepdim=True), (g.abs() * w).sum(1, keepdim=True)) if renormalize else (0.0, 0.0))
            qe = torch.gather(q, 1, e)
            want = want.scatter_add(1, e, routed_scale * w * (g - shift) * qe)
            bound = bound.scatter_add(1, e, abs(routed_scale) * w * (g.abs() + size) * qe * rel)
        dz = gradient(z, idx, start, k, alpha, sc, st, dloss, None if g is None else dw, renormalize=renormalize,
                      routed_scale=routed_scale)
        assert torch.isnan(dz[~inside]).all() and not dz[inside & ~live].any()
        err = ((dz.double() - want).abs() / (bound + 2 * U * want.abs() + 1e-37))[live]
        assert bool((err <= 1).all()), (float(err.max()), int((err > 1).sum()), int(err.argmax()) // E)


def routed(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)
    return z, torch.topk(z, k, dim=1).indices.to(torch.int32), torch.randn(T, k, generator=g), g


@pytest.mark.parametrize("T,E,k,start", [(1200, 64, 16, [200, 1200]), (262144, 16, 8, [700, 262144]),
                                         (200000, 24, 6, [5000, 100000, 200000]), (40000, 32, 16, [30000, 30000, 35000, 40000]),
                                         (5000, 512, 16, [4999, 5000]), (3000, 128, 9, [3000, 3000]), (150000, 8, 1, [149998, 150000])])
def test_tokens_before_the_first_sequence(T, E, k, start):
    """More of them than a block counts at once, ending inside its run, at its end and blocks further on."""
    z, idx, dw, _ = routed(T, E, k, T + k)
    check_large(z, idx, torch.tensor(start, dtype=torch.int32), dw, k)


@pytest.mark.parametrize("E,k", [(256, 6), (64, 8), (37, 3), (255, 12), (512, 16), (16, 2)])
@pytest.mark.parametrize("renormalize,scale", [(True, 1.0), (False, 2.5)])
def test_many_rows_a_warp(E, k, renormalize, scale):
    """Sequences of one to seven tokens, empty ones and long ones, tokens outside them all, padding at every place among
    a warp's tokens, dropped picks and experts picked twice."""
    T = 60000
    z, idx, dw, g = routed(T, E, k, E + k)
    short = 100 + torch.cumsum(torch.randint(0, 8, (4000,), generator=g), 0)
    start = torch.cat([torch.tensor([100]), short, torch.tensor([20000, 20000, 41111, T - 300])]).to(torch.int32)
    hit = lambda share: torch.rand(T, generator=g) < share  # noqa: E731
    if k > 1:
        idx[hit(0.1), k - 1] = E + 7
        idx[hit(0.05), k - 1] = -3
        twice = hit(0.1)
        idx[twice, 1] = idx[twice, 0]
    idx[hit(0.07), 0] = -1
    idx[30000:30400, 0] = -1
    check_large(z, idx, start, dw, k, renormalize=renormalize, routed_scale=scale)

"""Adapters and their gradients where every pipeline is full: many items for each block of the expand, many stages and
chunks of several tiles for the weights' gradients. All rows and all gradients against the float64 definition, computed
on the GPU, with the bounds of _finetune (derived there).
"""
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _finetune import HALF_BF16, SLACK, SUM, TINY, Pool
from test_gpu_lora import apply, backward

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()
    yield
    torch.cuda.empty_cache()


def expect(p):
    """{name: (value, bound)} of y, dx, dA and dB in float64 on the GPU."""
    x, dy, A, B, s, y, dx = (getattr(p, "d_" + v).double() for v in ("x", "dy", "A", "B", "scale", "y", "dx"))
    dA, dB, tA, tB = torch.zeros_like(A), torch.zeros_like(B), torch.zeros_like(A), torch.zeros_like(B)
    ty, tx = torch.zeros_like(y), torch.zeros_like(dx)
    for i in range(p.n):
        t = torch.nonzero(p.d_adapter == i)[:, 0]

        def low(v, W):  # value and error of s W v
            h = s[i] * (v @ W.T)
            return h, (W.shape[1] + 2) * SUM * s[i] * (v.abs() @ W.abs().T) + 2.0 ** -16 * h.abs()

        (h, eh), (g, eg) = low(x[t], A[i]), low(dy[t], B[i].T)
        last = (2 * p.R + 2) * SUM
        ty[t] = eh @ B[i].abs().T + last * (y[t].abs() + h.abs() @ B[i].abs().T)
        tx[t] = eg @ A[i].abs() + last * (dx[t].abs() + g.abs() @ A[i].abs())
        c = (2 * len(t) + 2) * SUM
        tA[i] = (eg + c * g.abs()).T @ x[t].abs()
        tB[i] = dy[t].abs().T @ (eh + c * h.abs())
        y[t] += h @ B[i].T
        dx[t] += g @ A[i]
        dA[i], dB[i] = g.T @ x[t], dy[t].T @ h
    return {k: (v, (HALF_BF16 * v.abs() + t) * SLACK + TINY) for k, v, t in (("y", y, ty), ("dx", dx, tx), ("dA", dA, tA), ("dB", dB, tB))}


def check(label, got, want):
    v, tol = want
    err = (got.double() - v).abs() / tol
    assert bool(torch.isfinite(got).all()) and float(err.max()) <= 1, (label, float(err.max()), int((err > 1).sum()))


def mixed(T, n, seed):
    """Long runs of one adapter, ragged short ones, tokens of any, and tokens of none."""
    g = torch.Generator().manual_seed(seed)
    a = torch.repeat_interleave(torch.randint(-1, n, (T,), generator=g), torch.randint(1, 900, (T,), generator=g))[:T].clone()
    a[T // 3: T // 2] = torch.randint(-1, n, (T // 2 - T // 3,), generator=g)
    short = torch.repeat_interleave(torch.randint(0, n, (T,), generator=g), torch.randint(1, 60, (T,), generator=g))
    a[T // 2: 2 * T // 3] = short[: 2 * T // 3 - T // 2]
    return a


# items of the expand for each of 152 blocks (y, dx) and tiles of a chunk of the weights' gradients
SHAPES = [(8192, 2048, 2048, 32, 6),     # 6.7, 6.7 and 7
          (4100, 1000, 4104, 72, 5),     # 6.9, 1.7 and 5
          (9000, 5000, 520, 128, 3),     # 2.3, 18 and 11
          (20000, 264, 1032, 8, 40),     # 9.2, 3.1 and 7, more tokens than the plan keeps in shared memory
          (6000, 2056, 3080, 56, 1)]     # 7.6, 5.1 and 7: one adapter


@pytest.mark.parametrize("T,K,N,R,n", SHAPES)
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_full_pipelines(T, K, N, R, n, order):
    adapter = mixed(T, n, T + R) if order == "mixed" else [(i * 2 * n) // T % n for i in range(T)]
    p = Pool(T, K, N, R, n, 19 * T + R, adapter).to(DEV)
    want = expect(p)
    y = apply(p, p.d_y)
    check("y", y, want["y"])
    inplace = p.d_y.clone()
    assert torch.equal(apply(p, inplace, inplace), y)
    dx, dA, dB = backward(p, p.d_dx)
    for label, v in (("dx", dx), ("dA", dA), ("dB", dB)):
        check(label, v, want[label])
    inplace = p.d_dx.clone()
    again = backward(p, inplace, inplace)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dA) and torch.equal(again[2], dB)
    _, a2, b2 = backward(p, None, None)
    assert torch.equal(a2, dA) and torch.equal(b2, dB)

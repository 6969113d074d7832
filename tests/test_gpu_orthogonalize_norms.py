"""Orthogonalised updates of matrices whose norm is far below eps: X = M / (|M| + eps) is tiny then, and keeps its digits
all the same. The bound is that of test_gpu_orthogonalize.py: what is kept and multiplied is a power of two times X, chosen
by X's size, so that roundings stay relative to it."""
import numpy as np
import pytest
import torch

from oracle import orthogonalize as oorth
from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _dense import STEPS, momentum, near
from _finetune import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMIT = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def run(m, steps, eps, scale=1.0):
    ws = torch.full((fb.flint_orthogonalize_workspace_bytes(*m.shape),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full(m.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    fb.flint_orthogonalize(m.to(DEV), out, steps, eps, ws, scale)
    assert fb.flint_moe_read_status(ws) == (fb.OK, 0)
    return out


def sized(m, norms):
    """The matrices of m with these norms."""
    return m * (torch.tensor(norms, dtype=torch.float64) / torch.linalg.matrix_norm(m.double())).float()[:, None, None]


# by products (few rows of long matrices, tiles, pairs of CTAs) and in one kernel (a cluster of four, of two, one CTA)
SHAPES = [(12, 9000), (9000, 12), (257, 515), (520, 256), (640, 640), (64, 2048), (128, 700), (16, 300)]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norms_below_eps(rows, cols):
    """From eps itself to 2^-90 of it in one batch, zeros among them. The result's size is a^5 |M| / eps."""
    eps = 1e-7
    ratios = [1.0, 0.3, 1e-2, 2e-3, 1e-4, 1e-6, 0.0, 1e-9, 1e-14, 2.0 ** -60, 2.0 ** -90]
    m = sized(momentum(len(ratios), rows, cols, rows, "noise"), [r * eps for r in ratios])
    got = run(m, STEPS, eps)
    for i, r in enumerate(ratios):
        near(got[i], oorth.orthogonalize(f64(m[i]), STEPS, eps), LIMIT, f"{r} eps")


@pytest.mark.parametrize("eps", [1e-38, 1e-45, 1e-3, 1e30])
def test_sizes_of_eps(eps):
    """eps at the ends of FP32, with norms of its size and a 64th of it (of 1e-30 beside the smallest, so that the values are
    FP32's normals)."""
    m = sized(momentum(2, 257, 515, 3, "noise"), [1.0, 1.0])
    m = torch.stack([m[0] * max(eps, 1e-30), m[1] * max(eps, 1e-30) / 64])
    got = run(m, STEPS, eps)
    for i in range(2):
        near(got[i], oorth.orthogonalize(f64(m[i]), STEPS, np.float32(eps)), LIMIT, f"matrix {i}")


@pytest.mark.parametrize("rows,cols", [(257, 515), (64, 600)])
@pytest.mark.parametrize("steps", [((1.5, -0.5, 0.0),) * 16, ((0.0, 1.0, 0.0),), ((0.25, 0.0, 0.0),) * 6, ((0.0, 200.0, -40.0), (3.4445, -4.775, 2.0315)),
                                   ((8.287, -23.596, 17.3), (4.107, -2.947, 0.545), (3.949, -2.909, 0.552), (3.318, -2.488, 0.51))])
def test_other_steps(rows, cols, steps):
    """Steps that grow slowly, that shrink, and that have no linear part, whose result is the cube's size. A step's S comes
    of three roundings and its P of one more of a whole, 2^-11 / sqrt(3) each: below 0.0012 of X for the cubes."""
    ratios = [1.0, 1e-2, 1e-5, 1e-8]
    m = sized(momentum(len(ratios), rows, cols, 9, "noise"), ratios)
    got = run(m, steps, 1.0, 2.0)
    for i, r in enumerate(ratios):
        near(got[i], oorth.orthogonalize(f64(m[i]), steps, 1.0, 2.0), LIMIT, f"{r} eps")

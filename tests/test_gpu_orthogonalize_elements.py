"""Orthogonalised updates value by value, where the norm of the error would hide a wrong corner, and by every kernel that
the products may take.

Bounds. A result's error is its own rounding, at most 2^-8 of the value, and what the steps' roundings leave: (1 + E) X
with E from many independent roundings, so that its values lie about zero with a root mean square below 0.003 of X's (see
test_gpu_orthogonalize.py). X's rows and columns here are alike (their entries come of the same normal numbers), so that a
single value of it stays below eight times that, 0.024 of the matrix's root mean square. The norm bound 2^-8 holds for any
thousand values and more, whose sums of squares are within a few per cent of their share.
"""
import numpy as np
import pytest
import torch

from oracle import orthogonalize as oorth
from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _dense import STEPS, momentum, near
from _dense_shapes import UPDATES_BY_PAIRS
from _finetune import HALF_BF16, check, f64
from _orthogonal import rounded, steps_error

pytestmark = pytest.mark.gpu
DEV = "cuda"
LIMIT = 2.0 ** -8
EPS = 1e-7


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def run(m):
    ws = torch.full((fb.flint_orthogonalize_workspace_bytes(*m.shape),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full(m.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    fb.flint_orthogonalize(m, out, STEPS, EPS, ws)
    assert fb.flint_moe_read_status(ws) == (fb.OK, 0)
    return out


def values(got, ref, label):
    near(got, ref, LIMIT, label)
    check(got, ref, HALF_BF16 * np.abs(ref) + 0.024 * np.sqrt(np.mean(ref * ref)), label)
    rows, cols = ref.shape
    for name, part in (("last rows", (slice(-32, None), slice(None))), ("last columns", (slice(None), slice(-32, None)))):
        if ref[part].size >= 1000:
            near(got[part], ref[part], LIMIT, f"{label} {name}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,rows,cols", UPDATES_BY_PAIRS)
def test_pairs_of_ctas(n, rows, cols, dtype):
    """Every product of a step by pairs of CTAs: triangles of tiles over a batch, values written twice, what the epilogue
    reads brought by TMA, last rows that TMA cannot reach."""
    m = momentum(n, rows, cols, rows + 1, "noise").to(dtype)
    got = run(m.to(DEV))
    for i in {0, 1, n // 2, n - 1}:
        values(got[i], oorth.orthogonalize(f64(m[i]), STEPS, EPS), f"matrix {i}")
    assert not got.isnan().any()
    assert torch.equal(run(m.to(DEV)), got)


# one tile a CTA (of both widths), clusters along K, few rows of long matrices, and the cluster kernel of every size
OTHERS = [(40, 140, 140), (80, 130, 140), (3, 300, 260), (1, 257, 515), (1, 515, 257), (1, 256, 2048), (1, 900, 2600), (1, 20, 9001),
          (1, 9001, 20), (2, 33, 700), (2, 700, 33), (5, 16, 1000), (2, 100, 1999), (1, 127, 2047), (1, 2047, 127)]


@pytest.mark.parametrize("n,rows,cols", OTHERS)
def test_other_kernels(n, rows, cols):
    m = momentum(n, rows, cols, cols + 1, "noise")
    got = run(m.to(DEV))
    for i in {0, n - 1}:
        values(got[i], oorth.orthogonalize(f64(m[i]), STEPS, EPS), f"matrix {i}")


@pytest.mark.parametrize("n,rows,cols", [(600, 65536, 64), (20000, 64, 2048)])
def test_the_last_of_many_alone(n, rows, cols):
    """The last matrix of a batch of more than 2^31 values, and the same matrix in a call of its own. Both are off from the
    exact result by less than 2^-8 of it."""
    assert n * rows * cols > 1 << 31
    gen = torch.Generator(DEV).manual_seed(n + 1)
    m = torch.randn(n, rows, cols, generator=gen, device=DEV)
    got = run(m)[n - 1].clone()
    last = m[n - 1:].clone()
    del m
    torch.cuda.empty_cache()
    alone = run(last)[0]
    ref = oorth.orthogonalize(f64(last[0]), STEPS, EPS)
    values(got, ref, "last")
    values(alone, ref, "alone")
    near(got, f64(alone), 2 * LIMIT, "both")


BIG_STEPS = ((8.287, -23.596, 17.3), (4.107, -2.947, 0.545), (3.949, -2.909, 0.552), (3.318, -2.488, 0.51))


@pytest.mark.parametrize("rows,cols", [(40, 600), (64, 600), (600, 64), (128, 600)])
def test_steps_of_large_coefficients(rows, cols):
    """Coefficients up to 24, whose P is larger than that of the usual steps and its roundings with it, and whose slopes
    carry errors on: below what _orthogonal derives from them, a bf16 rounding of a root mean square of 2^-8 / sqrt(3)
    beside it. (As it is with 40 rows, where slopes reach 30.)"""
    m = momentum(4, rows, cols, 9, "noise")
    m = (m / torch.linalg.matrix_norm(m)[:, None, None]).contiguous()
    ws = torch.full((fb.flint_orthogonalize_workspace_bytes(*m.shape),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full(m.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    fb.flint_orthogonalize(m.to(DEV), out, BIG_STEPS, 1.0, ws, 2.0)
    for i in range(4):
        limit = np.hypot(steps_error(f64(m[i]), BIG_STEPS, 1.0), HALF_BF16 / np.sqrt(3))
        near(out[i], oorth.orthogonalize(f64(m[i]), BIG_STEPS, 1.0, 2.0), limit, f"matrix {i}")


def alike(n, rows, cols, seed):
    """Matrices whose singular values lie within a fifth of one another: no averaging over them."""
    g = torch.Generator().manual_seed(seed)
    q = torch.linalg.qr(torch.randn(n, max(rows, cols), min(rows, cols), generator=g, dtype=torch.float64))[0]
    m = q * (0.8 + 0.4 * torch.rand(n, 1, min(rows, cols), generator=g))
    return (m if rows >= cols else m.transpose(1, 2)).float().contiguous()


@pytest.mark.parametrize("steps", [STEPS, BIG_STEPS])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (2, 2), (2, 30), (3, 4), (40, 3), (4, 4), (6, 60), (8, 8), (90, 8), (16, 500), (24, 40), (32, 32),
                                       (32, 2000), (3, 9000), (9000, 2), (16, 8200), (6200, 32)])
def test_few_rows_round_once(rows, cols, steps):
    """Up to 32 rows (or columns) the steps add next to nothing to the result's own rounding, whatever the singular values:
    |bf16(v + d) - v| <= |bf16(v) - v| + 2 |d|."""
    n = 30 if rows * cols < 5000 else 4
    for m in (momentum(n, rows, cols, rows, "noise"), alike(n, rows, cols, cols)):
        ws = torch.full((fb.flint_orthogonalize_workspace_bytes(*m.shape),), 0xFF, dtype=torch.uint8, device=DEV)
        out = torch.full(m.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
        fb.flint_orthogonalize(m.to(DEV), out, steps, EPS, ws)
        for i in range(n):
            ref = oorth.orthogonalize(f64(m[i]), steps, EPS)
            near(out[i], ref, rounded(ref) + 2 * steps_error(f64(m[i]), steps, EPS), f"matrix {i}")

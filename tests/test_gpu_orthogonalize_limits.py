"""Orthogonalised updates at the limits that the header states: the most matrices in a batch, the longest sides."""
import numpy as np
import pytest
import torch

from oracle import orthogonalize as oorth
from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _dense import STEPS, near
from _finetune import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-7


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def run(m):
    ws = torch.empty(fb.flint_orthogonalize_workspace_bytes(*m.shape), dtype=torch.uint8, device=DEV)
    out = torch.full(m.shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    fb.flint_orthogonalize(m, out, STEPS, EPS, ws)
    assert fb.flint_moe_read_status(ws) == (fb.OK, 0)
    return out


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (24, 17), (129, 130), (12, 8200)])
def test_most_matrices(rows, cols):
    """65535 matrices. One of a single row is its direction times what the steps make of one, the same for all: within
    2^-8 for the result's rounding and 2^-8 for the steps', whose roundings one row does not average."""
    n = 65535
    gen = torch.Generator(DEV).manual_seed(rows)
    m = torch.randn(n, rows, cols, generator=gen, device=DEV)
    got = run(m)
    assert not got.isnan().any()
    for i in (0, 1, 32767, 32768, n - 2, n - 1):
        near(got[i], oorth.orthogonalize(f64(m[i]), STEPS, EPS), 2.0 ** (-7 if rows == 1 else -8), f"matrix {i}")
    del m, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,cols", [(16384, 16384), (65536, 8), (8, 65536), (65536, 129), (129, 65535)])
def test_longest_sides(rows, cols):
    """Against the same steps in FP32 products, whose own error of 2^-23 a product, times the steps' growth of 485 in weak
    directions, is small beside the bound."""
    gen = torch.Generator(DEV).manual_seed(cols)
    m = torch.randn(1, rows, cols, generator=gen, device=DEV)
    got = run(m)[0]
    x = m[0] if rows <= cols else m[0].T
    x = (x / (torch.linalg.vector_norm(x.double()) + EPS).float()).contiguous()
    if min(rows, cols) < 200:
        x = x.double()
    for a, b, c in STEPS:
        s = x @ x.T
        x = a * x + (b * s + c * (s @ s)) @ x
    ref = x if rows <= cols else x.T
    err, size = torch.linalg.vector_norm(got.to(ref.dtype) - ref), torch.linalg.vector_norm(ref)
    assert float(err) <= 2.0 ** -8 * float(size)
    for part in ((slice(-64, None), slice(None)), (slice(None), slice(-64, None))):
        p = ref[part]
        assert float(torch.linalg.vector_norm(got[part].to(p.dtype) - p)) <= 2.0 ** -8 * float(torch.linalg.vector_norm(p))
    assert not torch.backends.cuda.matmul.allow_tf32 and np.isfinite(float(err))
    del m, got, x, ref
    torch.cuda.empty_cache()

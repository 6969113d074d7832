"""The orthogonalised update (through the C ABI) against the float64 definition.

The error's norm is below 2^-8 of the result's. The result's own rounding takes at most 2^-8 / sqrt(3) = 0.0023 of it in
the root mean square. X is kept to 22 bits. A step's S is off by three f16 roundings of at most 2^-11 / sqrt(3) = 2.8e-4
(its two factors and its own), its P by one more: with |b| s^2 + 2 |c| s^4 = 4.7 at s = 0.8 that is sqrt(3) 2.8e-4 * 4.7
and 2.8e-4 * 2.2 of X, together 0.0024 a step; errors of a step before come back with the polynomial's slope there, -0.3
to -0.7, so that all steps together stay below 0.003. The two together: 0.0038.
"""
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
EPS = 1e-7


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def run(m, steps=STEPS, eps=EPS, scale=1.0, out=None):
    """m on the device; [n][rows][cols] or one matrix."""
    shape = m.shape if m.dim() == 3 else (1, *m.shape)
    ws = torch.full((fb.flint_orthogonalize_workspace_bytes(*shape),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full(m.shape, float("nan"), dtype=torch.bfloat16, device=DEV) if out is None else out
    fb.flint_orthogonalize(m, out, steps, eps, ws, scale)
    assert fb.flint_moe_read_status(ws) == (fb.OK, 0)
    return out


def compare(m, got, **kw):
    for i in range(len(m)):
        near(got[i], oorth.orthogonalize(f64(m[i]), kw.get("steps", STEPS), EPS, kw.get("scale", 1.0)), LIMIT, f"matrix {i}")


# wide, square and tall; one row or column; sides that are no multiple of 8, 64 or 128; several matrices
SHAPES = [(1, 1, 1), (3, 1, 70), (2, 70, 1), (2, 8, 264), (5, 16, 1000), (3, 33, 129), (2, 129, 33), (1, 127, 128), (2, 128, 128), (1, 129, 130),
          (1, 64, 2048), (2, 2048, 64), (1, 256, 1024), (1, 300, 260), (1, 257, 515), (1, 640, 384), (3, 131, 131), (40, 24, 40),
          (90, 40, 100), (80, 100, 40), (21, 300, 260), (20, 260, 515), (20, 520, 257),
          (2, 16, 2048), (3, 2500, 24), (1, 64, 5120), (1, 5121, 64), (1, 128, 2048), (2, 1999, 127), (1, 100, 2049), (1, 9000, 12), (1, 900, 2600),
          (300, 20, 33)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,rows,cols", SHAPES)
def test_shapes(n, rows, cols, dtype):
    m = momentum(n, rows, cols, rows + cols).to(dtype)
    got = run(m.to(DEV))
    compare(m, got)
    assert torch.equal(run(m.to(DEV)), got)  # the same bits again
    if n > 1:  # a matrix does not depend on the others
        other = m.flip(0).to(DEV)
        other[n - 1] = m[n - 1].to(DEV)
        assert torch.equal(run(other)[n - 1], got[n - 1])
    if n > 1 and min(rows, cols) <= 64:  # nor on how many there are, where one kernel serves any number
        assert torch.equal(run(m[n - 1].to(DEV).contiguous()), got[n - 1])


@pytest.mark.parametrize("kind", ["noise", "spike"])
@pytest.mark.parametrize("rows,cols", [(64, 512), (300, 200), (256, 1024)])
def test_spectra(rows, cols, kind):
    m = momentum(1, rows, cols, 5, kind)
    compare(m, run(m.to(DEV)))


@pytest.mark.parametrize("power", [-120, -60, 60, 120])
def test_sizes_of_values(power):
    """The norm neither overflows nor vanishes: the result of 2^k M is that of M (eps apart, which counts beside small
    ones only)."""
    m = momentum(1, 40, 136, 6, "noise")
    got = run((m * 2.0 ** power).to(DEV), eps=1e-45)
    near(got[0], oorth.orthogonalize(f64(m[0]), STEPS, 0.0), LIMIT, f"2^{power}")


def test_zeros_and_eps():
    m = torch.zeros(3, 48, 72)
    m[1] = momentum(1, 48, 72, 7)[0]
    got = run(m.to(DEV))
    assert not got[0].any() and not got[2].any()
    compare(m[1:2], got[1:2])
    eps = float(torch.linalg.matrix_norm(m[1]))  # halves X
    near(run(m[1].to(DEV), eps=eps), oorth.orthogonalize(f64(m[1]), STEPS, eps), LIMIT, "eps")


def test_other_steps_and_scale():
    m = momentum(2, 96, 200, 8)
    one = ((1.5, -0.5, 0.0),)  # the cubic step
    for steps, scale in ((one, 1.0), (one * 16, -2.0), (((8.287, -23.596, 17.3), (4.107, -2.947, 0.545), (3.949, -2.909, 0.552)), 0.25),
                         (((0.0, 0.0, 0.0),), 1.0)):
        got = run(m.to(DEV), steps=steps, scale=scale)
        compare(m, got, steps=steps, scale=scale)


def test_in_place_and_no_matrices():
    m = momentum(2, 40, 264, 9).to(torch.bfloat16)
    a = m.to(DEV)
    want = run(a)
    assert run(a, out=a) is a and torch.equal(a, want)
    none = torch.empty(0, 4, 4, device=DEV)
    fb.flint_orthogonalize(none, none.bfloat16(), STEPS, EPS, torch.empty(256, dtype=torch.uint8, device=DEV))


def test_streams_and_graphs():
    ms = [momentum(2, 100, 260, s).to(DEV) for s in (1, 2)]
    want = [run(m) for m in ms]
    torch.cuda.synchronize()
    got = []
    for m in ms:
        with torch.cuda.stream(torch.cuda.Stream()):
            got.append(run(m))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(fb.flint_orthogonalize_workspace_bytes(2, 100, 260), dtype=torch.uint8, device=DEV)
    src, out = ms[0].clone(), torch.empty(2, 100, 260, dtype=torch.bfloat16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.flint_orthogonalize(src, out, STEPS, EPS, ws)
    for m, w in zip(ms[::-1], want[::-1]):
        src.copy_(m)
        out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(out, w)


def test_singular_values():
    """What the steps are for: singular values near one, the directions kept."""
    m = momentum(1, 192, 640, 10, "noise")
    got = f64(run(m.to(DEV))[0])
    s = np.linalg.svd(got, compute_uv=False)
    assert 0.6 < s.min() and s.max() < 1.3

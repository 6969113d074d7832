"""Low-rank rows that leave BF16's range: infinite ones, and finite ones above its largest value, which the two halves
that enter the second product have to carry (through the C ABI)."""
import numpy as np
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _finetune import HALF_BF16, Pool, f64
from test_gpu_lora import apply, backward

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def signs(n):
    return torch.tensor([1.0, -1.0, -1.0]).repeat(n // 3 + 1)[:n]


@pytest.mark.parametrize("T", [6, 31, 150])
@pytest.mark.parametrize("R", [8, 24, 64, 72])
def test_infinite_low_rank_values(T, R):
    """One token's x holds an infinity: its low-rank row is infinite, all of one sign, and so are the outputs that B's
    signs make; nothing else changes. The same for dy, g and dx, and for the gradients that such rows enter."""
    K, N, n, bad = 136, 200, 2, 4
    adapter = [t % n for t in range(T)]
    p = Pool(T, K, N, R, n, 7 * T + R, adapter)
    p.A[:, :, 3] = p.A[:, :, 3].abs() + 0.125      # h = +infinity in every rank
    p.B[:] = (p.B.abs() + 0.125) * signs(N)[None, :, None]
    p.to(DEV)
    clean_y = apply(p, p.d_y)
    p.d_x[bad, 3] = float("inf")
    y = apply(p, p.d_y)
    rest = torch.arange(T, device=DEV) != bad
    assert torch.equal(y[rest], clean_y[rest])
    assert torch.equal(y[bad].float().cpu(), signs(N) * float("inf"))
    # dB = sum dy h: infinite with dy's sign for that adapter
    _, _, dB = backward(p, p.d_dx)
    assert torch.equal(dB[bad % n].float().cpu(), (p.dy[bad].float().sign() * float("inf"))[:, None].expand(N, R))

    p.A[:] = (p.A.abs() + 0.125) * signs(K)
    p.B[:, 5] = p.B[:, 5].abs()                      # g = +infinity in every rank
    p.to(DEV)
    clean = backward(p, p.d_dx)
    p.d_dy[bad, 5] = float("inf")
    dx, dA, dB = backward(p, p.d_dx)
    assert torch.equal(dx[rest], clean[0][rest])
    assert torch.equal(dx[bad].float().cpu(), signs(K) * float("inf"))
    assert torch.equal(dA[bad % n].float().cpu(), (p.x[bad].float().sign() * float("inf")).expand(R, K))
    other = 1 - bad % n
    assert torch.equal(dA[other], clean[1][other]) and torch.equal(dB[other], clean[2][other])


@pytest.mark.parametrize("T", [5, 32, 140])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_low_rank_values_above_the_largest_bf16(T, sign):
    """h = 1.99957 2^127 is finite in FP32 and lies above the largest BF16 value; B's 2^-20 bring it back. Two roundings
    to 16 bits and one to bf16 are allowed."""
    K, N, R, n = 64, 72, 8, 1
    p = Pool(T, K, N, R, n, 3, [0] * T)
    for v in (p.A, p.B, p.x, p.y, p.dy, p.dx):
        v.zero_()
    p.scale[:] = 1.0
    m = 181 / 128  # its square is 1.99957
    p.A[0, 2, 1] = m * 2.0 ** 63
    p.x[:, 1] = sign * m * 2.0 ** 64
    p.B[0, :, 2] = 2.0 ** -20
    p.to(DEV)
    y = f64(apply(p, None))
    want = sign * m * m * 2.0 ** 107
    assert np.all(np.abs(y - want) <= abs(want) * (HALF_BF16 + 2.0 ** -16)), y
    p.dy[:, 4] = 2.0 ** -20
    p.to(DEV)
    dB = f64(backward(p, None)[2])
    want_b = T * want
    assert np.all(np.abs(dB[0, 4, 2] - want_b) <= abs(want_b) * (HALF_BF16 + 2.0 ** -16 + T * 2.0 ** -23))
    # g likewise
    p.B.zero_()
    p.B[0, 4, 2] = m * 2.0 ** 63
    p.dy[:, 4] = sign * m * 2.0 ** 64
    p.A[0, 2, :] = 2.0 ** -20
    p.x.zero_()
    p.x[:, 7] = 2.0 ** -20
    p.to(DEV)
    dx, dA, _ = backward(p, None)
    assert np.all(np.abs(f64(dx) - want) <= abs(want) * (HALF_BF16 + 2.0 ** -16))
    assert np.all(np.abs(f64(dA)[0, 2, 7] - want_b) <= abs(want_b) * (HALF_BF16 + 2.0 ** -16 + T * 2.0 ** -23))

"""The dense gated block at its limits: gates far below zero."""
import numpy as np
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _finetune import HALF_BF16, SUM, check, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def ws_of(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)


def nans(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("T", [40, 1300])
def test_gates_far_below_zero(T):
    """silu where e^-g is near FP32's largest value, or above it: g e^g is still a value of its own, which a large u brings
    back. Tokens lie along two axes, so that g, u and y come of one product each, without a sum's rounding. The exponential
    is off by 2 + 1.2 |g| steps of 2^-23 (and, below FP32's normals, by 2^-149: 2^-19 of e^-90), its quotient and the
    products by six more; h and y are rounded to bf16."""
    H, I = 8, 2600
    gates = torch.tensor([-84.0, -86.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0]).repeat(I // 8)
    gate, up, down = torch.zeros(I, H), torch.zeros(I, H), torch.zeros(H, I)
    gate[:, 0], up[:, 1] = gates, 2.0 ** 100
    for n in range(H):  # y[n] = h at the begin, the end and a place between
        down[n, (n, 8 * 200 + n, I - 8 + n)[n % 3]] = 1.0
    x = torch.zeros(T, H)
    x[:, 0], x[:, 1] = 1.0, 2.0 ** (torch.arange(T) % 7 - 3).float()
    d = [v.bfloat16().to(DEV) for v in (x, gate, up, down)]
    f = fb.flint_ffn_init(*d[1:])
    y = nans(T, H)
    fb.flint_ffn_forward(f, d[0], T, y, ws_of(fb.flint_ffn_workspace_bytes(f, T)))
    g = f64(gates[:8])
    ref = (g * np.exp(g) / (1 + np.exp(g)))[None, :] * 2.0 ** 100 * f64(d[0])[:, 1:2]
    check(y, ref, np.abs(ref) * ((2 + 1.2 * np.abs(g) + 6) * SUM + 2.0 ** -19 + 2 * HALF_BF16 + HALF_BF16 ** 2), "y")

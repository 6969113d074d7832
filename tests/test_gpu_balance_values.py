"""Values at which the router's gradient loses digits if its sums are not arranged for them (bounds of
test_gpu_balance.py).
"""
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _finetune import router
from test_gpu_balance import check_all, gradient

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


@pytest.mark.parametrize("k,big", [(3, 1e4), (8, 1e4), (12, 1e5), (3, -1e6)])
def test_a_large_gradient_of_an_unlikely_pick(k, big):
    """A pick of a small weight whose gradient dwarfs the others' leaves those their digits, wherever it stands."""
    E, T = 16, 3 * k
    z, idx, start, dw = router(T, E, k, 40 + k, [0, T])
    for t in range(T):
        j = t % k  # its place among the picks
        z[t, int(idx[t, j])] = -14.0
        dw[t, j] = big
    z[0], idx[0], dw[0] = 0.0, torch.arange(k, dtype=torch.int32), 1.0
    z[0, :3] = torch.tensor([-14.0, 1.0, 0.0])
    dw[0, :3] = torch.tensor([big, 1.0, 2.0])
    check_all(z, idx, start, dw, k)


@pytest.mark.parametrize("E,k", [(2, 1), (32, 4), (130, 3), (36, 12)])
def test_rows_of_very_low_scores(E, k):
    """Rows of logits from -10 down to -90 with experts that are masked or far below the rest: their shares are those
    of the definition, and a masked expert's gradient is exactly zero."""
    T = 40
    z, _, start, dw = router(T, E, k, 50 + E, [0, T])
    z[:] = 0.25 * z - torch.linspace(10.0, 90.0, T)[:, None]
    z[1::3, E - 1] = -float("inf")
    z[26:36:3, 0] = -95.0  # rows of -62 and below
    z[27:36:3, 0] = torch.finfo(torch.float32).min
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
    _, sc, st = check_all(z, idx, start, dw, k)
    for g in (None, dw):
        assert not gradient(z, idx, start, k, 0.5, sc, st, 1e20, g)[1::3, E - 1].any()


def test_a_masked_expert_beside_ordinary_scores():
    """Picked or not, in a row of any size: zero."""
    z, idx, start, dw = router(30, 64, 4, 60, [0, 30])
    z[::2, 5] = z[::2, 40] = -float("inf")
    idx[::4, 1] = 5
    _, sc, st = check_all(z, idx, start, dw, 4)
    dz = gradient(z, idx, start, 4, 0.5, sc, st, 1e38, dw)
    assert not dz[::2, 5].any() and not dz[::2, 40].any()

"""Values at which the router's gradient loses digits if its sums are not arranged for them (bounds of
test_gpu_balance.py).
"""
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _finetune import router
from test_gpu_balance import check_all

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

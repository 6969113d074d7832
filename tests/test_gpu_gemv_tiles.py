"""The dense GEMV's choice between one tile a block (or cluster) and several: at every border of the choice each row has
the bits of the call for that row alone, and the choice may be made first inside a capture."""
import os
import subprocess
import sys

import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300 import layers
from w4a16_moe_decode_gb300.build import build

from test_gpu_gemv_rows import test_adapters_beside_split_rows as adapters_beside

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


# Blocks of four warps (K of no multiple of 512) around four an SM; clusters of 2, 3 and 4 around what runs at once,
# in one round, in several, and in rounds that are mostly empty.
@pytest.mark.parametrize("N,K", [(9728, 256), (9744, 256), (12000, 768), (9744, 1280), (6080, 1792), (7312, 1792),
                                 (3648, 4096), (3712, 4096), (5600, 4096), (1552, 6144), (3200, 6144), (1200, 8192), (3648, 8192)])
@pytest.mark.parametrize("fmt", [fb.NVFP4, fb.BF16])
@pytest.mark.parametrize("B", [1, 2, 7, 32])
def test_rows_equal_single_calls(N, K, fmt, B):
    packed, _ = layers.synth_dense(N, K, 9, 0, fmt, DEV)
    x = layers.synth_x(B, K, 9, 0, DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = torch.full((B, N), 0x7FC0, dtype=torch.int16, device=DEV)
    fb.flint_gemv(packed, N, K, fmt, x, B, y, None, 1e-6, status)
    for t in (0, B // 2, B - 1):
        one = torch.full((1, N), 0x7FC0, dtype=torch.int16, device=DEV)
        fb.flint_gemv(packed, N, K, fmt, x[t:t + 1], 1, one, None, 1e-6, status)
        assert torch.equal(one[0], y[t]), t
    assert int(status.item()) == 0
    # the tiles' sums do not depend on how many tiles there are: the first ones, packed alone
    few = 64
    part, _ = layers.synth_dense(few, K, 9, 0, fmt, DEV)
    alone = torch.full((B, few), 0x7FC0, dtype=torch.int16, device=DEV)
    fb.flint_gemv(part, few, K, fmt, x, B, alone, None, 1e-6, status)
    if fmt == fb.BF16:  # (an NVFP4 matrix' scale is its own largest value's)
        assert torch.equal(alone, y[:, :few])


@pytest.mark.parametrize("B,K,N,R,n,fmt", [(1, 4096, 512, 16, 2, fb.NVFP4), (1, 8192, 1168, 40, 1, fb.NVFP4), (1, 8192, 272, 24, 3, fb.BF16),
                                           (1, 6144, 2000, 8, 1, fb.BF16), (1, 6144, 3200, 16, 2, fb.BF16), (3, 1280, 9760, 16, 2, fb.NVFP4),
                                           (6, 768, 9760, 24, 3, fb.BF16)])
def test_adapters_beside_each_choice(B, K, N, R, n, fmt):
    """One tile a cluster for one row, with room for the next call and without; blocks of four warps with several tiles."""
    adapters_beside(B, K, N, R, n, fmt)


@pytest.mark.parametrize("N,K,fmt", [(512, 4096, fb.NVFP4), (1168, 8192, fb.NVFP4), (2000, 6144, fb.BF16)])
def test_one_normalised_row_has_the_bits_of_any_batch(N, K, fmt):
    packed, _ = layers.synth_dense(N, K, 11, 0, fmt, DEV)
    x, g = layers.synth_x(5, K, 11, 0, DEV), layers.synth_norm(K, 11, 0, DEV)
    y = torch.full((5, N), 0x7FC0, dtype=torch.int16, device=DEV)
    fb.flint_gemv(packed, N, K, fmt, x, 5, y, g, 1e-6)
    for t in range(5):
        one = torch.full((1, N), 0x7FC0, dtype=torch.int16, device=DEV)
        fb.flint_gemv(packed, N, K, fmt, x[t:t + 1], 1, one, g, 1e-6)
        assert torch.equal(one[0], y[t]), t


FIRST = """
import sys
sys.path[:0] = [{root!r}]
import torch
from w4a16_moe_decode_gb300 import binding as fb, layers
cases = []
for N, K, fmt, B in ((2560, 4096, fb.BF16, 1), (3200, 6144, fb.NVFP4, 5), (2400, 8192, fb.BF16, 20)):
    packed, _ = layers.synth_dense(N, K, 1, 0, fmt, "cuda")
    cases.append((packed, N, K, fmt, B, layers.synth_x(B, K, 1, 0, "cuda"), torch.zeros(B, N, dtype=torch.bfloat16, device="cuda")))
def step():
    for packed, N, K, fmt, B, x, y in cases:
        fb.flint_gemv(packed, N, K, fmt, x, B, y)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
first = [c[-1].clone() for c in cases]
for c in cases:
    c[-1].zero_()
step()
torch.cuda.synchronize()
assert all(v.any() and torch.equal(v, c[-1]) for v, c in zip(first, cases))
print("captured first")
"""


def test_first_calls_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "captured first" in res.stdout, res.stderr[-2000:]

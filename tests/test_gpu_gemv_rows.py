"""The dense GEMV for many tiles, whose blocks stage their rows once for several tiles: every row's
sums have the order that calls of up to eight rows use, so the results are the same bits; and with adapters beside it
(their bound as in test_gpu_lora.py)."""
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300 import layers
from w4a16_moe_decode_gb300.build import build

from test_gpu_lora import SLACK, SUM, check, f64, gemv_case, gemv_lora

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


@pytest.mark.parametrize("N,K,fmt", [(2464, 2048, fb.NVFP4), (2448, 768, fb.BF16), (2464, 4096, fb.NVFP4), (2480, 4096, fb.BF16),
                                     (1360, 8192, fb.NVFP4), (2064, 6144, fb.NVFP4), (16, 4096, fb.NVFP4)])
@pytest.mark.parametrize("B", [9, 13, 16, 17, 24, 25, 32])
@pytest.mark.parametrize("norm", [False, True])
def test_rows_equal_calls_of_eight(N, K, fmt, B, norm):
    packed, _ = layers.synth_dense(N, K, 7, 0, fmt, DEV)
    x = layers.synth_x(B, K, 7, 0, DEV)
    g = layers.synth_norm(K, 7, 0, DEV) if norm else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(rows):
        y = torch.full((rows.shape[0], N), 0x7FC0, dtype=torch.int16, device=DEV)
        fb.flint_gemv(packed, N, K, fmt, rows, rows.shape[0], y, g, 1e-6, status)
        return y

    want = torch.cat([run(x[i:i + 8]) for i in range(0, B, 8)])
    got = run(x)
    assert torch.equal(got, want) and int(status.item()) == 0


@pytest.mark.parametrize("B,K,N,R,n,fmt", [(13, 4096, 2464, 32, 5, fb.NVFP4), (32, 6144, 1360, 16, 3, fb.NVFP4),
                                           (20, 4096, 1296, 64, 20, fb.BF16)])
def test_adapters_beside_split_rows(B, K, N, R, n, fmt):
    p, packed, W = gemv_case(B, K, N, R, n, fmt, 170 + B)
    x = f64(p.x)
    ref, tol = p.expect_apply(x @ W.T)
    # the base's FP32 sum over K, and its f16 rows: x / max|x| is exact down to 2^-24 of its largest value
    tol = tol + SLACK * ((K + 4) * SUM * (abs(x) @ abs(W).T) + 2.0 ** -24 * abs(x).max(1)[:, None] * abs(W).sum(1)[None, :])
    y = gemv_lora(p, packed, fmt)
    check(y, ref, tol, "gemv_lora")
    assert torch.equal(gemv_lora(p, packed, fmt), y)


@pytest.mark.parametrize("B,K,N,R,n,fmt", [(1, 2048, 4992, 8, 1, fb.NVFP4), (8, 512, 5008, 24, 2, fb.NVFP4), (3, 768, 4928, 16, 3, fb.BF16),
                                           (1, 4096, 2464, 16, 2, fb.NVFP4), (5, 8192, 1360, 40, 5, fb.NVFP4),
                                           (8, 6144, 1040, 8, 1, fb.BF16)])
def test_few_rows_of_many_tiles(B, K, N, R, n, fmt):
    """Parity, and the bits of each row alone."""
    test_adapters_beside_split_rows(B, K, N, R, n, fmt)
    packed, _ = layers.synth_dense(N, K, 7, 0, fmt, DEV)
    x = layers.synth_x(B, K, 7, 0, DEV)
    for g in (None, layers.synth_norm(K, 7, 0, DEV)):
        y = torch.full((B, N), 0x7FC0, dtype=torch.int16, device=DEV)
        fb.flint_gemv(packed, N, K, fmt, x, B, y, g, 1e-6)
        for t in range(B):
            one = torch.full((1, N), 0x7FC0, dtype=torch.int16, device=DEV)
            fb.flint_gemv(packed, N, K, fmt, x[t:t + 1], 1, one, g, 1e-6)
            assert torch.equal(one[0], y[t]), t

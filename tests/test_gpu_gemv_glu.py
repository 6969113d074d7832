"""The gated pair of projections for decode (through the C ABI) against the float64 definition.

Bounds, derived before any run (see _dense for the terms): the weights c are exact, the activations lose at most 2^-25 of
their row's largest value in their f16 form (NVFP4), which adds 2^-25 max|x| sum|c| G to a product:
    |dg| = ((K + 2) 2^-23 |x||c| + 2^-25 max|x| sum|c|) G,   |dh| = 1.1 |dg||u| + |silu(g)||du| + (2^-8 + FN) |h|
"""
import numpy as np
import pytest
import torch

import synth
from oracle import ffn as offn
from oracle import moe, nvfp4
from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300 import layers
from w4a16_moe_decode_gb300.build import build

from _common import bits_to_f64
from _dense import FN
from _finetune import HALF_BF16, SLACK, SUM, TINY, check

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def matrices(I, K, seed, fmt):
    """(gate, up): the oracle's matrix and the canonical source of each."""
    out = []
    for tag in (synth.GATE, synth.UP):
        w = synth.matrix_f32(seed, 0, tag, 0, I, K, 0.02)
        if fmt == fb.NVFP4:
            codes, scales, G = nvfp4.quantize(w)
            src = {"codes": torch.from_numpy(np.ascontiguousarray(codes)).to(DEV), "scales": torch.from_numpy(np.ascontiguousarray(scales)).to(DEV),
                   "global": torch.full((1,), float(G), device=DEV)}
            out.append((moe.NVFP4Matrix(codes, scales, G), src))
        else:
            bits = synth.f32_to_bf16_bits(w)
            out.append((moe.BF16Matrix(bits), {"bf16": torch.from_numpy(bits.view(np.int16)).to(DEV)}))
    return out


def pack(mats, I, K, fmt):
    dst = torch.full((fb.flint_gemv_glu_packed_bytes(I, K, fmt),), 0xFF, dtype=torch.uint8, device=DEV)
    fb.flint_gemv_glu_pack(mats[0][1], mats[1][1], I, K, fmt, dst)
    return dst


def expect(x, mats, fmt):
    gc, uc = (np.float64(m.G) * m.c() for m, _ in mats)
    g, u = x @ gc.T, x @ uc.T
    h = offn.hidden(g, u)
    loss = 2.0 ** -25 * np.abs(x).max(1, keepdims=True) if fmt == fb.NVFP4 else 0.0
    eg, eu = ((x.shape[1] + 2) * SUM * (np.abs(x) @ np.abs(c).T) + loss * np.abs(c).sum(1) for c in (gc, uc))
    eh = 1.1 * eg * np.abs(u) + np.abs(g * offn.sigmoid(g)) * eu + (HALF_BF16 + FN) * np.abs(h)
    return h, eh * SLACK + TINY


def run(I, K, B, seed, fmt, norm=False, rows=None):
    mats = matrices(I, K, seed, fmt)
    packed = pack(mats, I, K, fmt)
    x = layers.synth_x(B, K, seed, 0, DEV)
    w = layers.synth_norm(K, seed, 0, DEV) if norm else None
    h = torch.full((B + 1, I), float("nan"), dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    fb.flint_gemv_glu(packed, I, K, fmt, x, B, h, w, 1e-6, status)
    assert int(status.item()) == 0 and h[B].isnan().all()
    xo = bits_to_f64(x)
    if norm:
        xo = moe.rmsnorm(xo, moe.bf16_bits_to_f64(synth.norm_bf16(seed, 0, K)), 1e-6)
    rows = list(range(B)) if rows is None else rows
    check(h[:B][rows], *expect(xo[rows], mats, fmt), f"glu I={I} K={K} B={B}")
    return packed, x, h[:B], w


@pytest.mark.parametrize("fmt", [fb.NVFP4, fb.BF16])
@pytest.mark.parametrize("I,K,B", [(8, 256, 1), (40, 256, 5), (136, 512, 8), (64, 768, 9), (72, 1280, 17), (256, 2048, 32), (64, 1792, 24)])
def test_one_tile_a_block(I, K, B, fmt):
    run(I, K, B, 70 + B, fmt)


@pytest.mark.parametrize("fmt", [fb.NVFP4, fb.BF16])
@pytest.mark.parametrize("I,K,B", [(2600, 512, 3), (5008, 256, 1), (2560, 768, 14), (2608, 256, 20), (2472, 1024, 32)])
def test_several_tiles_a_block(I, K, B, fmt):
    run(I, K, B, 80 + B, fmt, rows=[0, B - 1])


@pytest.mark.parametrize("I,K,B,norm", [(1304, 2048, 17, False), (1304, 2048, 32, True), (2472, 2048, 25, False), (1600, 1536, 32, False)])
def test_two_groups_a_block(I, K, B, norm):
    """Rows that fill an SM: two groups of warps, each with its own tiles."""
    run(I, K, B, 110 + B, fb.NVFP4, norm, rows=[0, B // 2, B - 1])


@pytest.mark.parametrize("fmt", [fb.NVFP4, fb.BF16])
@pytest.mark.parametrize("I,K,B,norm", [(16, 4096, 1, False), (40, 8192, 2, True), (24, 6144, 9, False), (32, 4096, 32, True),
                                        (1400, 4096, 1, False), (1304, 8192, 3, True), (1208, 4096, 16, False), (1000, 4096, 27, False)])
def test_split_over_a_cluster(I, K, B, norm, fmt):
    run(I, K, B, 90 + B, fmt, norm, rows=[0, B - 1])


@pytest.mark.parametrize("fmt", [fb.NVFP4, fb.BF16])
@pytest.mark.parametrize("I,K,B", [(128, 1024, 4), (96, 768, 17), (2600, 256, 6)])
def test_norm_prologue(I, K, B, fmt):
    run(I, K, B, 100 + B, fmt, norm=True)


@pytest.mark.parametrize("I,K", [(64, 512), (2600, 256), (48, 4096), (1304, 2048)])
def test_a_row_stands_alone(I, K):
    """A row's bits do not depend on the other rows of the call."""
    packed, x, h, _ = run(I, K, 32, 7, fb.NVFP4, rows=[0])
    for B in (1, 8, 20):
        part = torch.empty(B, I, dtype=torch.bfloat16, device=DEV)
        fb.flint_gemv_glu(packed, I, K, fb.NVFP4, x, B, part)
        assert torch.equal(part, h[:B])


def test_pack_reports_nan_scales():
    mats = matrices(16, 256, 3, fb.NVFP4)
    dst = torch.empty(fb.flint_gemv_glu_packed_bytes(16, 256), dtype=torch.uint8, device=DEV)
    for m, want in ((None, 0), (0, fb.DEV_ERR_NAN_SCALE), (1, fb.DEV_ERR_NAN_SCALE)):
        src = [{k: v.clone() for k, v in s.items()} for _, s in mats]
        if m is not None:
            src[m]["scales"].view(-1)[37] = 0x7F
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        fb.flint_gemv_glu_pack(src[0], src[1], 16, 256, fb.NVFP4, dst, st)
        assert int(st.item()) == want


def test_gemv_of_two_groups_has_the_rows_of_smaller_calls():
    """flint_gemv with 17 to 32 rows of 2048, more tiles than blocks: the bits of calls of fewer rows."""
    N, K = 2608, 2048
    packed, _ = layers.synth_dense(N, K, 5, 0, fb.NVFP4, DEV)
    x = layers.synth_x(32, K, 5, 0, DEV)
    y = torch.empty(32, N, dtype=torch.int16, device=DEV)
    for B in (17, 24, 25, 32):
        y.fill_(0x7FC0)
        fb.flint_gemv(packed, N, K, fb.NVFP4, x, B, y)
        for r in (0, 8, B - 1):
            one = torch.empty(1, N, dtype=torch.int16, device=DEV)
            fb.flint_gemv(packed, N, K, fb.NVFP4, x[r : r + 1].contiguous(), 1, one)
            assert torch.equal(one[0], y[r]), (B, r)
        assert bool((y[B:] == 0x7FC0).all())

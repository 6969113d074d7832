"""Refusals of the balance loss and its gradient for buffers that overlap, without a GPU."""
import ctypes

import pytest

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return fb.lib()


T, E, K, SEQS = 2000, 64, 6, 3
FORWARD = dict(z=0x1000000, idx=0x2000000, seq=0x3000000, loss=0x4000000, c=0x4100000, sc=0x4200000, st=0x4300000, w=0x4400000)
BACKWARD = dict(z=0x1000000, idx=0x2000000, seq=0x3000000, sc=0x4200000, st=0x4300000, dl=0x4500000, dw=0x4600000, dz=0x6000000)
SIZES = dict(z=4 * T * E, idx=4 * T * K, seq=4 * (SEQS + 1), loss=4, c=4 * E, sc=4 * SEQS * E, st=4 * SEQS, dl=4, dw=4 * T * K, dz=4 * T * E)


def forward(lib, cfg, z, idx, seq, loss, c, sc, st, w):
    return lib.flint_moe_balance(ctypes.byref(cfg), z, idx, T, seq, SEQS, 0.1, loss, c, sc, st, w, 1 << 20, None)


def backward(lib, cfg, z, idx, seq, sc, st, dl, dw, dz):
    return lib.flint_moe_balance_backward(ctypes.byref(cfg), z, idx, T, seq, SEQS, 0.1, sc, st, dl, dw, dz, None)


@pytest.mark.parametrize("call,base,outs", [(forward, FORWARD, ("loss", "c", "sc", "st", "w")), (backward, BACKWARD, ("dz",))])
def test_outputs_lie_apart(lib, call, base, outs):
    cfg = fb.make_config(num_experts=E, top_k=K)
    sizes = dict(SIZES, w=fb.flint_moe_balance_workspace_bytes(cfg, T, SEQS))
    for out in outs:
        for other in base:
            if other == out:
                continue
            places = [base[other]]
            if out not in ("w", "dz"):  # (those are aligned to 16 bytes)
                places.append(base[other] + sizes[other] - 4)
            elif sizes[other] > 16:
                places.append(base[other] + (sizes[other] - 4) // 16 * 16)
            for at in places:
                assert call(lib, cfg, **dict(base, **{out: at})) == fb.EINVAL, (out, other, at)


def test_one_sequence_has_counts_of_its_own(lib):
    """counts and seq_counts have the same shape then, but not the same memory."""
    cfg = fb.make_config(num_experts=E, top_k=K)
    assert lib.flint_moe_balance(ctypes.byref(cfg), 0x1000000, 0x2000000, T, None, 1, 0.1, 0x4000000, 0x4100000, 0x4100000, 0x4300000,
                                 0x4400000, 1 << 20, None) == fb.EINVAL

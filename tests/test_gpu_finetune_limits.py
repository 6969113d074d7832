"""The fine-tuning operators at their limits: rows farther apart than 32 bits reach, more picks times experts than 32
bits hold, and first calls that a graph captures."""
import os
import subprocess
import sys

import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _finetune import Pool
from test_gpu_balance import U, cfg_of
from test_gpu_lora import apply, backward, ws_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()
    yield
    torch.cuda.empty_cache()


def apart(v, ld):
    """The rows of v, ld elements apart."""
    rows, cols = v.shape
    out = torch.empty((rows - 1) * ld + cols, dtype=v.dtype, device=DEV).as_strided((rows, cols), (ld, 1))
    return out.copy_(v)


@pytest.mark.parametrize("T,ld,run", [(20, 1 << 27, 1), (200, 1 << 24, 1), (200, 1 << 24, 70)])
def test_rows_past_32_bits(T, ld, run):
    K, N, R, n = 136, 264, 16, 3
    p = Pool(T, K, N, R, n, 40 + T, [(t // run) % (n + 1) - 1 for t in range(T)]).to(DEV)
    want_y, want = apply(p, p.d_y), backward(p, p.d_dx)
    assert (T - 1) * ld > 1 << 31
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    x, y = apart(p.d_x, ld), apart(p.d_y, ld)
    fb.flint_lora_apply(lora, x, p.d_adapter, T, y, y, ws_of(fb.flint_lora_workspace_bytes(lora, T)))
    assert torch.equal(y, want_y)
    del y
    dy, dx = apart(p.d_dy, ld), apart(p.d_dx, ld)
    dA, dB = torch.empty_like(p.d_A), torch.empty_like(p.d_B)
    fb.flint_lora_backward(lora, x, dy, p.d_adapter, T, dx, dx, dA, dB, ws_of(fb.flint_lora_backward_workspace_bytes(lora, T)))
    assert torch.equal(dx, want[0]) and torch.equal(dA, want[1]) and torch.equal(dB, want[2])


def test_loads_past_32_bits():
    """k T E above 2^31: the loads' whole numbers need 64 bits. Bounds as in test_gpu_balance.py."""
    T, E, k, alpha = 300_000, 512, 16, 0.5
    assert k * T * E > 1 << 31
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn(T, E, generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
    cfg = cfg_of(E, k)
    loss, dz = torch.empty(1, device=DEV), torch.empty_like(z)
    counts, sc, st = (torch.empty(s, dtype=torch.int32, device=DEV) for s in ((E,), (1, E), (1,)))
    fb.flint_moe_balance(cfg, z, idx, T, None, 1, alpha, loss, counts, sc, st,
                         ws_of(fb.flint_moe_balance_workspace_bytes(cfg, T, 1)))
    fb.flint_moe_balance_backward(cfg, z, idx, T, None, 1, alpha, sc, st, None, None, dz)
    c = torch.bincount(idx.flatten().long(), minlength=E)
    assert torch.equal(counts.long(), c) and torch.equal(sc[0].long(), c) and int(st) == T
    f1 = (E * c - k * T).double() / (k * T)
    s = torch.sigmoid(z.double())
    p = s / s.sum(1, keepdim=True)
    F = p @ f1
    ref = float(alpha * (1 + F).mean())
    r = (4 * float(z.abs().max()) + 16) * U
    assert abs(float(loss) - ref) <= (r + (E / 16 + 16) * U) * (abs(ref) + alpha)
    q = torch.sigmoid(-z.double())
    want = alpha / T * p * (f1 - F[:, None]) * q
    tol = alpha / T * p * q * (f1.abs() + (p @ f1.abs())[:, None]) * (4 * r + (E / 8 + 32) * U) + 2 * U * want.abs() + 1e-37
    assert bool(((dz - want).abs() <= tol).all())


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from w4a16_moe_decode_gb300 import binding as fb, layers
from _finetune import Pool
ps = [Pool(T, 256, 256, 16, 3, T).to("cuda") for T in (12, 150)]
packed, _ = layers.synth_dense(256, 256, 1, 0, fb.NVFP4, "cuda")
cfg = fb.make_config(hidden=256, num_experts=16, top_k=2, inter=64)
cases = []
for T in (100, 4000):
    z = torch.randn(T, 16, device="cuda")
    cases.append((z, torch.topk(z, 2, dim=1).indices.to(torch.int32)))
ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
outs = []
def step():
    for p in ps:
        lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
        y, dx, dA, dB = (torch.zeros_like(v) for v in (p.d_y, p.d_dx, p.d_A, p.d_B))
        fb.flint_lora_apply(lora, p.d_x, p.d_adapter, p.T, p.d_y, y, ws)
        fb.flint_lora_backward(lora, p.d_x, p.d_dy, p.d_adapter, p.T, p.d_dx, dx, dA, dB, ws)
        outs.extend((y, dx, dA, dB))
    p, y = ps[0], torch.zeros_like(ps[0].d_y)
    fb.flint_gemv_lora(packed, 256, 256, fb.NVFP4, p.d_x, p.T, y, fb.flint_lora_init(p.d_A, p.d_B, p.d_scale), p.d_adapter, ws)
    outs.append(y)
    for z, idx in cases:
        T = z.shape[0]
        loss, dz = torch.zeros(1, device="cuda"), torch.zeros_like(z)
        c, sc, st = (torch.zeros(s, dtype=torch.int32, device="cuda") for s in ((16,), (1, 16), (1,)))
        fb.flint_moe_balance(cfg, z, idx, T, None, 1, 0.1, loss, c, sc, st, ws)
        fb.flint_moe_balance_backward(cfg, z, idx, T, None, 1, 0.1, sc, st, None, None, dz)
        outs.extend((loss, c, dz))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
first = [v.clone() for v in outs]
outs.clear()
step()
torch.cuda.synchronize()
assert len(first) == len(outs) and all(torch.equal(a, b) for a, b in zip(first, outs))
print("captured first")
"""


def test_first_calls_inside_a_capture():
    tests = os.path.dirname(os.path.abspath(__file__))
    script = FIRST.format(root=os.path.dirname(tests), tests=tests)
    res = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and "captured first" in res.stdout, res.stderr[-2000:]

"""The dense block's operators as they are used together: a training step (forward, gradients, orthogonalised updates), the
adapters' and the router's updates, and the updated weights served by the decode calls."""
import os
import subprocess
import sys

import pytest
import torch

from oracle import ffn as offn
from oracle import orthogonalize as oorth
from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _dense import STEPS, Block, near
from _finetune import Pool, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def ws_of(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)


def test_training_step_then_decode():
    """Against the same step in float64, each stage on what the stage before gave: 2^-8 of the norm for one or two
    roundings to bf16 (see test_gpu_ffn.py, test_gpu_orthogonalize.py)."""
    T, H, I, lr = 200, 256, 512, 0.05
    p = Block(T, H, I, 4).to(DEV)
    f = fb.flint_ffn_init(p.d_gate, p.d_up, p.d_down)
    ws = ws_of(fb.flint_ffn_backward_workspace_bytes(f, T))
    y, g, u = torch.empty_like(p.d_x), torch.empty_like(p.d_g), torch.empty_like(p.d_u)
    fb.flint_ffn_forward(f, p.d_x, T, y, ws, g, u)
    dx, grads = torch.empty_like(p.d_x), [torch.empty_like(v) for v in (p.d_gate, p.d_up, p.d_down)]
    fb.flint_ffn_backward(f, p.d_x, g, u, p.d_dy, T, dx, *grads, ws)
    refs = offn.backward(*(f64(v) for v in (p.x, g, u, p.dy, p.gate, p.up, p.down)))
    near(dx, refs[0], 2.0 ** -8, "dx")
    pair = torch.stack(grads[:2])  # gate and up as one batch
    ups = torch.empty_like(pair)
    fb.flint_orthogonalize(pair, ups, STEPS, 1e-7, ws_of(fb.flint_orthogonalize_workspace_bytes(2, I, H)))
    down = torch.empty_like(grads[2])
    fb.flint_orthogonalize(grads[2], down, STEPS, 1e-7, ws_of(fb.flint_orthogonalize_workspace_bytes(1, H, I)))
    for got, grad, ref in zip((*ups, down), grads, refs[1:]):
        near(grad, ref, 2.0 ** -8, "gradient")
        near(got, oorth.orthogonalize(f64(grad), STEPS, 1e-7), 2.0 ** -8, "update")
    for w, d in zip((p.d_gate, p.d_up, p.d_down), (*ups, down)):
        w.sub_(lr * d)  # the handle's weights are updated where they lie
    fb.flint_ffn_forward(f, p.d_x, T, y, ws)
    want, _, _ = offn.forward(*(f64(v) for v in (p.x, p.d_gate, p.d_up, p.d_down)))
    near(y, want, 2.0 ** -8, "y of the updated weights")
    # the same weights packed for decode
    B = 9
    packed = ws_of(fb.flint_gemv_glu_packed_bytes(I, H, fb.BF16))
    fb.flint_gemv_glu_pack({"bf16": p.d_gate}, {"bf16": p.d_up}, I, H, fb.BF16, packed)
    pdown = ws_of(fb.flint_gemv_packed_bytes(H, I, fb.BF16))
    fb.flint_gemv_pack({"bf16": p.d_down}, H, I, fb.BF16, pdown)
    h, yd = torch.empty(B, I, dtype=torch.bfloat16, device=DEV), torch.empty(B, H, dtype=torch.bfloat16, device=DEV)
    fb.flint_gemv_glu(packed, I, H, fb.BF16, p.d_x, B, h)
    fb.flint_gemv(pdown, H, I, fb.BF16, h, B, yd)
    near(yd, want[:B], 2.0 ** -8, "decode")


def test_updates_of_adapters_and_router():
    """flint_lora_backward's gradients, orthogonalised adapter by adapter (an adapter without tokens stays as it is), and
    a router's."""
    p = Pool(300, 256, 192, 16, 4, 5, [t % 3 for t in range(300)]).to(DEV)
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    dA, dB = torch.empty_like(p.d_A), torch.empty_like(p.d_B)
    fb.flint_lora_backward(lora, p.d_x, p.d_dy, p.d_adapter, 300, None, None, dA, dB, ws_of(fb.flint_lora_backward_workspace_bytes(lora, 300)))
    for d in (dA, dB):
        out = torch.empty_like(d)
        fb.flint_orthogonalize(d, out, STEPS, 1e-7, ws_of(fb.flint_orthogonalize_workspace_bytes(*d.shape)), 0.2)
        assert not out[3].any()
        for i in range(3):
            near(out[i], oorth.orthogonalize(f64(d[i]), STEPS, 1e-7, 0.2), 2.0 ** -8, "adapter")
    dz = torch.randn(500, 16, device=DEV) / 500  # a router's gradient of its logits
    dw = dz.T @ torch.randn(500, 256, device=DEV)
    out = torch.empty(16, 256, dtype=torch.bfloat16, device=DEV)
    fb.flint_orthogonalize(dw, out, STEPS, 1e-7, ws_of(fb.flint_orthogonalize_workspace_bytes(1, 16, 256)))
    near(out, oorth.orthogonalize(f64(dw), STEPS, 1e-7), 2.0 ** -8, "router")


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from w4a16_moe_decode_gb300 import binding as fb
from _dense import STEPS, Block, momentum
blocks = [Block(T, H, I, T).to("cuda") for T, H, I in ((40, 256, 264), (1400, 264, 1704))]
mats = [momentum(n, r, c, r).to("cuda") for n, r, c in ((2, 16, 300), (2, 64, 600), (3, 100, 2000), (1, 300, 500), (30, 300, 260))]
ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
bf = [torch.randn(s, device="cuda").bfloat16() for s in ((64, 256), (64, 256))]
packed = torch.empty(fb.flint_gemv_glu_packed_bytes(64, 256, fb.BF16), dtype=torch.uint8, device="cuda")
outs = []
def step():
    for p in blocks:
        f = fb.flint_ffn_init(p.d_gate, p.d_up, p.d_down)
        y, g, u, dx = (torch.zeros_like(v) for v in (p.d_x, p.d_g, p.d_u, p.d_x))
        dw = [torch.zeros_like(v) for v in (p.d_gate, p.d_up, p.d_down)]
        fb.flint_ffn_forward(f, p.d_x, p.T, y, ws, g, u)
        fb.flint_ffn_backward(f, p.d_x, g, u, p.d_dy, p.T, dx, *dw, ws)
        outs.extend((y, g, u, dx, *dw))
    for m in mats:
        o = torch.zeros(m.shape, dtype=torch.bfloat16, device="cuda")
        fb.flint_orthogonalize(m, o, STEPS, 1e-7, ws)
        outs.append(o)
    h = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    fb.flint_gemv_glu_pack(dict(bf16=bf[0]), dict(bf16=bf[1]), 64, 256, fb.BF16, packed)
    fb.flint_gemv_glu(packed, 64, 256, fb.BF16, blocks[0].d_x, 3, h)
    outs.append(h)
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


@pytest.mark.parametrize("n,rows,cols", [(600, 65536, 64), (20000, 64, 2048)])
def test_batches_past_32_bits(n, rows, cols):
    """More than 2^31 values in a batch: the last matrix as the definition has it, and as it is alone in the norm."""
    assert n * rows * cols > 1 << 31
    gen = torch.Generator(DEV).manual_seed(n)
    m = torch.randn(n, rows, cols, generator=gen, device=DEV)
    out = torch.empty(n, rows, cols, dtype=torch.bfloat16, device=DEV)
    fb.flint_orthogonalize(m, out, STEPS, 1e-7, ws_of(fb.flint_orthogonalize_workspace_bytes(n, rows, cols)))
    last = m[n - 1].clone()
    near(out[n - 1], oorth.orthogonalize(f64(last), STEPS, 1e-7), 2.0 ** -8, "last")
    near(out[n // 2 + 1], oorth.orthogonalize(f64(m[n // 2 + 1]), STEPS, 1e-7), 2.0 ** -8, "middle")
    del m, out
    torch.cuda.empty_cache()


def test_updates_beside_a_decode_on_another_stream():
    """An update and the decode calls of other weights at the same time, on two streams with their own workspaces."""
    p = Block(12, 256, 512, 11).to(DEV)
    packed = ws_of(fb.flint_gemv_glu_packed_bytes(512, 256, fb.BF16))
    fb.flint_gemv_glu_pack({"bf16": p.d_gate}, {"bf16": p.d_up}, 512, 256, fb.BF16, packed)
    m = torch.randn(2, 512, 700, device=DEV)
    ws = ws_of(fb.flint_orthogonalize_workspace_bytes(2, 512, 700))

    def both(a, b):
        o, h = torch.empty(2, 512, 700, dtype=torch.bfloat16, device=DEV), torch.empty(12, 512, dtype=torch.bfloat16, device=DEV)
        fb.flint_orthogonalize(m, o, STEPS, 1e-7, ws, stream=a)
        for _ in range(4):
            fb.flint_gemv_glu(packed, 512, 256, fb.BF16, p.d_x, 12, h, stream=b)
        return o, h

    want = both(None, None)
    torch.cuda.synchronize()
    got = both(torch.cuda.Stream(), torch.cuda.Stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))

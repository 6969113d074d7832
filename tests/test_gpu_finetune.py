"""The fine-tuning operators as they are used together: a routed layer's router gradient with its balance loss, and
adapters beside a packed projection in serving and in a training step.
"""
import numpy as np
import pytest
import torch

from oracle import balance as ob
from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300 import layers
from w4a16_moe_decode_gb300.build import build

from _common import TINY
from _finetune import SLACK, SUM, Pool, check, f64
from test_gpu_balance import check_all
from test_gpu_lora import gemv_case, gemv_lora, ws_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def test_router_gradient_of_a_routed_layer():
    """The expert-grouped path routes a batch; its logits and picks go through the balance loss and its gradient, and
    the counts agree with the picks."""
    cfg = fb.make_config(**TINY)
    T, E, k = 90, cfg.num_experts, cfg.top_k
    dl = layers.synth_layer(cfg, 21, 0, DEV)
    x = layers.synth_x(T, cfg.hidden, 5, 0, DEV)
    out = torch.empty_like(x)
    ws = layers.prefill_workspace(cfg, T, DEV)
    fb.flint_moe_prefill(dl.handle, x, T, out, ws)
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    logits = torch.empty(T, E, device=DEV)
    fb.flint_moe_prefill_debug_routing(cfg, ws, T, idx, w, logits)
    torch.cuda.synchronize()
    start = torch.tensor([0, 31, 31, T], dtype=torch.int32)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    _, sc, _ = check_all(logits.cpu(), idx.cpu(), start, dw, k)
    assert int(sc.sum()) == T * k


@pytest.mark.parametrize("B", [3, 32])
def test_serving_step_equals_training_forward(B):
    """The decode form (projection and adapters in one rounding) and the many-token form on the projection's own output
    are both within their bounds of the same sum; then a training step's gradients of the same adapters move them and
    the decode form follows."""
    D, R, n = 512, 16, 3
    p, packed, W = gemv_case(B, D, D, R, n, fb.NVFP4, 200 + B)
    base = f64(p.x) @ W.T
    ref, tol = p.expect_apply(base)
    gtol = SLACK * ((D + 4) * SUM * (np.abs(f64(p.x)) @ np.abs(W).T)
                    + 2.0 ** -24 * np.abs(f64(p.x)).max(1)[:, None] * np.abs(W).sum(1)[None, :])
    y = gemv_lora(p, packed, fb.NVFP4)
    check(y, ref, tol + gtol, "decode form")
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    y2 = torch.empty_like(y)
    fb.flint_gemv(packed, D, D, fb.NVFP4, p.d_x, B, y2)
    proj = f64(y2)
    fb.flint_lora_apply(lora, p.d_x, p.d_adapter, B, y2, y2, ws_of(fb.flint_lora_workspace_bytes(lora, B)))
    check(y2, *p.expect_apply(proj), "projection, then adapters in place")

    refs, tols = p.expect_backward()
    dx, dA, dB = torch.empty_like(p.d_dx), torch.empty_like(p.d_A), torch.empty_like(p.d_B)
    fb.flint_lora_backward(lora, p.d_x, p.d_dy, p.d_adapter, B, p.d_dx, dx, dA, dB,
                           ws_of(fb.flint_lora_backward_workspace_bytes(lora, B)))
    for v, r, t, label in zip((dx, dA, dB), refs, tols, ("dx", "dA", "dB")):
        check(v, r, t, label)
    p.d_A.sub_(0.125 * dA)  # an update in place: the pool's pointers stay
    p.d_B.sub_(0.125 * dB)
    p.A, p.B = p.d_A.cpu(), p.d_B.cpu()
    ref, tol = p.expect_apply(base)
    check(gemv_lora(p, packed, fb.NVFP4), ref, tol + gtol, "decode form after an update")


def test_a_whole_step_in_one_graph():
    """Projection with adapters, its gradients, the router's loss and gradient, captured once and replayed: the same
    bits as the calls made one by one."""
    D, R, n, T, E, k = 256, 8, 4, 200, 16, 2
    p = Pool(T, D, D, R, n, 77).to(DEV)
    cfg = fb.make_config(**TINY)
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(3)).to(DEV)
    idx = torch.topk(z, k, dim=1).indices.to(torch.int32)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(4)).to(DEV)
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    new = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731

    def buffers():
        return dict(y=new(T, D), dx=new(T, D), dA=torch.zeros_like(p.d_A), dB=torch.zeros_like(p.d_B),
                    loss=new(1, dtype=torch.float32), counts=new(E, dtype=torch.int32), sc=new(1, E, dtype=torch.int32),
                    st=new(1, dtype=torch.int32), dz=new(T, E, dtype=torch.float32))

    wl = ws_of(max(fb.flint_lora_workspace_bytes(lora, T), fb.flint_lora_backward_workspace_bytes(lora, T)))
    wb = ws_of(fb.flint_moe_balance_workspace_bytes(cfg, T, 1))

    def step(o):
        fb.flint_lora_apply(lora, p.d_x, p.d_adapter, T, p.d_y, o["y"], wl)
        fb.flint_moe_balance(cfg, z, idx, T, None, 1, 0.01, o["loss"], o["counts"], o["sc"], o["st"], wb)
        fb.flint_moe_balance_backward(cfg, z, idx, T, None, 1, 0.01, o["sc"], o["st"], None, dw, o["dz"])
        fb.flint_lora_backward(lora, p.d_x, p.d_dy, p.d_adapter, T, p.d_dx, o["dx"], o["dA"], o["dB"], wl)

    a, b = buffers(), buffers()
    step(a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        step(b)
    for _ in range(2):
        for v in b.values():
            v.fill_(1)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a[key], b[key]) for key in a)
    assert fb.flint_moe_read_status(wl) == (fb.OK, 0)
    assert abs(float(a["loss"]) - ob.loss(f64(z), idx.cpu().numpy(), [0, T], k, 0.01)) <= 40 * 2.0 ** -24 * 0.01  # (4 |z| + 16 + E / 16) u of alpha, |z| < 5

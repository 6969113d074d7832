"""The dense gated block at its limits: more saved values than 32 bits count, long runs of k-blocks in the gradients, gates
far below zero."""
import numpy as np
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _dense import Block, near
from _dense_shapes import LONG
from _finetune import HALF_BF16, SUM, check, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("dx", "dgate", "dup", "ddown")


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


@pytest.mark.parametrize("T,H,I", LONG)
def test_gradients_of_long_runs(T, H, I):
    p = Block(T, H, I, 5 * T + I).to(DEV)
    refs, tols = p.expect_backward()
    f = fb.flint_ffn_init(p.d_gate, p.d_up, p.d_down)
    ws = ws_of(fb.flint_ffn_backward_workspace_bytes(f, T))
    got = [nans(T, H)] + [nans(*v.shape) for v in (p.gate, p.up, p.down)]
    fb.flint_ffn_backward(f, p.d_x, p.d_g, p.d_u, p.d_dy, T, *got, ws)
    assert fb.flint_moe_read_status(ws) == (fb.OK, 0)
    for v, ref, tol, label in zip(got, refs, tols, NAMES):
        check(v, ref, tol, label)
        near(v, ref, 2.0 ** -8, label)


def test_saved_values_past_32_bits():
    """65536 tokens of 8 x 65536: 2^32 values of g and of u. The definition in float64 on the device, in chunks of tokens;
    error norms below 2^-8 as in test_gpu_ffn.py, of all of each result and of the last tokens and columns."""
    T, H, I = 65536, 8, 65536
    assert T * I > 1 << 31
    gen = torch.Generator(DEV).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    x, dy = rnd(T, H).bfloat16(), rnd(T, H).bfloat16()
    gate, up, down = (rnd(I, H) * H ** -0.5).bfloat16(), (rnd(I, H) * H ** -0.5).bfloat16(), (rnd(H, I) * I ** -0.5).bfloat16()
    f = fb.flint_ffn_init(gate, up, down)
    y, g, u = nans(T, H), nans(T, I), nans(T, I)
    ws = torch.empty(fb.flint_ffn_backward_workspace_bytes(f, T), dtype=torch.uint8, device=DEV)
    fb.flint_ffn_forward(f, x, T, y, ws, g, u)
    assert fb.flint_moe_read_status(ws) == (fb.OK, 0)
    dx, dw = nans(T, H), [nans(I, H), nans(I, H), nans(H, I)]
    fb.flint_ffn_backward(f, x, g, u, dy, T, dx, *dw, ws)
    assert fb.flint_moe_read_status(ws) == (fb.OK, 0)
    wg, wu, wd = gate.double(), up.double(), down.double()
    sums = [torch.zeros(I, H, dtype=torch.float64, device=DEV) for _ in range(2)] + [torch.zeros(H, I, dtype=torch.float64, device=DEV)]
    off = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    step = 2048
    for t in range(0, T, step):
        xs, ds, s = x[t:t + step].double(), dy[t:t + step].double(), slice(t, t + step)
        ge, ue = xs @ wg.T, xs @ wu.T
        assert off(g[s], ge) <= 2.0 ** -8 and off(u[s], ue) <= 2.0 ** -8
        assert off(g[s][:, -64:], ge[:, -64:]) <= 2.0 ** -8 and off(u[s][:, -64:], ue[:, -64:]) <= 2.0 ** -8
        assert off(y[s], (ge * torch.sigmoid(ge) * ue) @ wd.T) <= 2.0 ** -8
        ge, ue = g[s].double(), u[s].double()  # the gradients are those of the saved values
        sg = torch.sigmoid(ge)
        dh = ds @ wd
        dg, du = dh * ue * sg * (1 + ge * (1 - sg)), dh * ge * sg
        assert off(dx[s], dg @ wg + du @ wu) <= 2.0 ** -8
        sums[0] += dg.T @ xs
        sums[1] += du.T @ xs
        sums[2] += ds.T @ (ge * sg * ue)
        del ge, ue, sg, dh, dg, du
    for got, ref in zip(dw, sums):
        assert off(got, ref) <= 2.0 ** -8
    assert off(dw[0][-64:], sums[0][-64:]) <= 2.0 ** -8 and off(dw[2][:, -64:], sums[2][:, -64:]) <= 2.0 ** -8
    del g, u, ws, sums
    torch.cuda.empty_cache()

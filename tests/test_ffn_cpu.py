"""Definitions of the dense block and of the orthogonalised update, and what their entry points refuse (without a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import ffn as offn
from oracle import orthogonalize as oorth
from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _dense import STEPS, Block, momentum
from _finetune import f64


@pytest.fixture(scope="module")
def lib():
    build()
    return fb.lib()


def test_definition_against_autograd():
    p = Block(17, 24, 40, 1)
    w = [torch.tensor(f64(v), requires_grad=True) for v in (p.x, p.gate, p.up, p.down)]
    x, gate, up, down = w
    g, u = x @ gate.T, x @ up.T
    y = (torch.nn.functional.silu(g) * u) @ down.T
    ref, g64, u64 = offn.forward(*(f64(v) for v in (p.x, p.gate, p.up, p.down)))
    assert np.allclose(ref, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    y.backward(torch.tensor(f64(p.dy)))
    got = offn.backward(f64(p.x), g64, u64, f64(p.dy), *(f64(v) for v in (p.gate, p.up, p.down)))
    for a, b in zip(got, w):
        assert np.allclose(a, b.grad.numpy(), rtol=1e-12, atol=1e-12)


def test_definition_against_differences():
    p = Block(5, 16, 24, 2)
    args = [f64(v) for v in (p.x, p.gate, p.up, p.down)]
    dy = f64(p.dy)
    _, g, u = offn.forward(*args)
    grads = offn.backward(args[0], g, u, dy, *args[1:])
    rng = np.random.default_rng(0)
    for i, (v, grad) in enumerate(zip(args, grads)):
        d = rng.standard_normal(v.shape)
        side = [(dy * offn.forward(*args[:i], v + e * d, *args[i + 1:])[0]).sum() for e in (1e-5, -1e-5)]
        assert abs((side[0] - side[1]) / 2e-5 - (grad * d).sum()) <= 1e-7 * np.abs(grad * d).sum()


@pytest.mark.parametrize("rows,cols", [(6, 20), (20, 6), (9, 9), (1, 5)])
def test_steps_against_the_products(rows, cols):
    m = momentum(1, rows, cols, 3)[0].double()
    x = m / (torch.linalg.matrix_norm(m) + 1e-7)
    for a, b, c in STEPS:
        s = x @ x.T
        x = a * x + (b * s + c * s @ s) @ x
    assert np.allclose(oorth.orthogonalize(m.numpy(), STEPS, 1e-7), x.numpy(), rtol=1e-9, atol=1e-11)


def handle(H=256, I=512):
    f = fb.flint_ffn()
    st = fb.lib().flint_ffn_init(H, I, 0x10000000, 0x20000000, 0x30000000, ctypes.byref(f))
    return st, f


def test_ffn_handle(lib):
    assert handle()[0] == fb.OK
    for H, I in ((0, 8), (12, 8), (8, 4), (65544, 8), (8, 65544), (-8, 8)):
        assert handle(H, I)[0] == fb.EUNSUPPORTED
    f = fb.flint_ffn()
    for args, want in (((256, 512, None, 0x20000000, 0x30000000), fb.EINVAL), ((256, 512, 0x10000008, 0x20000000, 0x30000000), fb.EALIGN),
                       ((256, 512, 0x10000000, 0x20000000, None), fb.EINVAL)):
        assert lib.flint_ffn_init(*args, ctypes.byref(f)) == want
    assert lib.flint_ffn_init(256, 512, 0x10000000, 0x20000000, 0x30000000, None) == fb.EINVAL
    _, f = handle()
    for T, ok in ((0, False), (1, True), (65536, True), (65537, False), (-1, False)):
        assert (fb.flint_ffn_workspace_bytes(f, T) > 0) == ok and (fb.flint_ffn_backward_workspace_bytes(f, T) > 0) == ok
    sizes = [fb.flint_ffn_workspace_bytes(f, T) for T in range(1, 400)]
    back = [fb.flint_ffn_backward_workspace_bytes(f, T) for T in range(1, 400)]
    assert sizes == sorted(sizes) and back == sorted(back)  # a workspace serves every smaller call


def test_ffn_forward_refusals(lib):
    _, f = handle()
    def call(f=f, x=0x40000000, ldx=256, T=40, y=0x50000000, ldy=256, g=None, u=None, w=0x60000000, nb=1 << 20):
        return lib.flint_ffn_forward(ctypes.byref(f), x, ldx, T, y, ldy, g, u, w, nb, None)
    assert call(T=0) == fb.OK and call(T=0, x=None, y=None, w=None, nb=0) == fb.OK
    for kw in (dict(T=-1), dict(T=65537), dict(x=None), dict(y=None), dict(w=None), dict(nb=256), dict(ldx=248), dict(ldy=128),
               dict(ldx=1 << 31), dict(ldy=1 << 31), dict(g=0x70000000), dict(u=0x70000000), dict(y=0x40000000), dict(y=0x40000010),
               dict(y=0x10000000), dict(g=0x70000000, u=0x70000000), dict(g=0x40000000, u=0x70000000),
               dict(g=0x70000000, u=0x60000000), dict(w=0x40000000), dict(w=0x30000000), dict(w=0x50000000)):
        assert call(**kw) == fb.EINVAL, kw
    for kw in (dict(x=0x40000008), dict(y=0x50000008), dict(w=0x60000010), dict(ldx=260), dict(ldy=260),
               dict(g=0x70000002, u=0x71000000)):
        assert call(**kw) == fb.EALIGN, kw
    assert lib.flint_ffn_forward(None, 0x40000000, 256, 1, 0x50000000, 256, None, None, 0x60000000, 1 << 20, None) == fb.EINVAL


def test_ffn_backward_refusals(lib):
    _, f = handle()
    def call(x=0x40000000, ldx=256, g=0x41000000, u=0x42000000, dy=0x43000000, lddy=256, T=40, dx=0x44000000, lddx=256,
             a=0x50000000, b=0x51000000, c=0x52000000, w=0x60000000, nb=1 << 20):
        return lib.flint_ffn_backward(ctypes.byref(f), x, ldx, g, u, dy, lddy, T, dx, lddx, a, b, c, w, nb, None)
    assert call(T=0, a=None, b=None, c=None) == fb.OK and call(dx=None, a=None, b=None, c=None) == fb.OK
    for kw in (dict(T=-1), dict(T=65537), dict(x=None), dict(g=None), dict(u=None), dict(dy=None), dict(w=None), dict(nb=1024),
               dict(ldx=8), dict(lddy=8), dict(lddx=8), dict(lddx=1 << 31), dict(a=None), dict(b=None), dict(c=None),
               dict(a=None, b=None), dict(dx=0x40000000), dict(dx=0x43000000), dict(dx=0x41000000), dict(a=0x51000000),
               dict(c=0x10000000), dict(b=0x44000000), dict(w=0x41000000), dict(w=0x52000000)):
        assert call(**kw) == fb.EINVAL, kw
    for kw in (dict(x=0x40000002), dict(g=0x41000008), dict(u=0x42000004), dict(dy=0x43000008), dict(dx=0x44000008), dict(a=0x50000008),
               dict(b=0x51000004), dict(c=0x52000002), dict(w=0x60000080), dict(ldx=258), dict(lddy=260), dict(lddx=260)):
        assert call(**kw) == fb.EALIGN, kw


def test_gemv_glu_refusals(lib):
    for I, K, ok in ((8, 256, True), (12, 256, False), (0, 256, False), (1 << 19, 256, True), ((1 << 19) + 8, 256, False),
                     (64, 4096, True), (64, 3200, False), (64, 128, False)):
        assert (fb.flint_gemv_glu_packed_bytes(I, K) > 0) == ok, (I, K)
    assert fb.flint_gemv_glu_packed_bytes(64, 256, 7) == 0
    def call(p=0x10000000, I=64, K=256, fmt=fb.NVFP4, x=0x20000000, B=4, h=0x30000000, n=None, eps=0.0):
        return lib.flint_gemv_glu(p, I, K, fmt, x, B, h, n, ctypes.c_float(eps), None, None)
    assert call(B=0) == fb.OK
    for kw in (dict(B=33), dict(B=-1), dict(p=None), dict(x=None), dict(h=None), dict(eps=-1.0), dict(eps=float("nan"))):
        assert call(**kw) == fb.EINVAL, kw
    for kw in (dict(I=12), dict(K=300), dict(fmt=3)):
        assert call(**kw) == fb.EUNSUPPORTED, kw
    for kw in (dict(p=0x10000008), dict(x=0x20000002), dict(h=0x30000008), dict(n=0x40000008)):
        assert call(**kw) == fb.EALIGN, kw
    s = fb.flint_gemv_src(0x10000000, 0x11000000, 0x12000000, None)
    none = fb.flint_gemv_src(None, 0x11000000, 0x12000000, None)
    def pack(g=s, u=s, I=64, dst=0x20000000, nb=1 << 20):
        return lib.flint_gemv_glu_pack(ctypes.byref(g) if g else None, ctypes.byref(u) if u else None, I, 256, fb.NVFP4, dst, nb, None, None)
    for kw in (dict(g=None), dict(u=None), dict(g=none), dict(u=none), dict(dst=None), dict(nb=64)):
        assert pack(**kw) == fb.EINVAL, kw
    assert pack(I=20) == fb.EUNSUPPORTED and pack(dst=0x20000008) == fb.EALIGN


def test_orthogonalize_refusals(lib):
    size = lib.flint_orthogonalize_workspace_bytes
    for n, r, c, ok in ((1, 1, 1, True), (0, 4, 4, False), (1, 0, 4, False), (1, 4, 0, False), (65535, 4, 4, True), (65536, 4, 4, False),
                        (1, 65536, 8, True), (1, 65537, 8, False), (1, 16384, 16384, True), (1, 16385, 16385, False)):
        assert (size(n, r, c) > 0) == ok, (n, r, c)
    def call(m=0x10000000, fmt=0, n=2, r=64, c=96, co=(1.0, -0.5, 0.1), steps=1, eps=1e-7, scale=1.0, out=0x20000000, w=0x30000000,
             nb=1 << 24):
        arr = None if co is None else (ctypes.c_float * len(co))(*co)
        return lib.flint_orthogonalize(m, fmt, n, r, c, arr, steps, ctypes.c_float(eps), ctypes.c_float(scale), out, w, nb, None)
    assert call(n=0) == fb.OK
    inf, nan = float("inf"), float("nan")
    for kw in (dict(m=None), dict(out=None), dict(w=None), dict(co=None), dict(steps=0), dict(steps=17), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=nan), dict(eps=inf), dict(scale=nan), dict(scale=inf), dict(co=(1.0, nan, 0.0)), dict(co=(1.0, 0.0, inf)),
               dict(nb=4096), dict(out=0x10000000), dict(out=0x10000010), dict(fmt=1, out=0x10000010), dict(w=0x10000000), dict(w=0x20000000), dict(m=0x30000100)):
        assert call(**kw) == fb.EINVAL, kw
    for kw in (dict(fmt=2), dict(r=0), dict(c=-1), dict(r=65537), dict(n=-1), dict(n=65536)):
        assert call(**kw) == fb.EUNSUPPORTED, kw
    for kw in (dict(m=0x10000008), dict(out=0x20000002), dict(w=0x30000010)):
        assert call(**kw) == fb.EALIGN, kw


def test_binding_refuses_other_shapes_and_types():
    f, b = torch.float32, torch.bfloat16
    gate, up, down = (torch.zeros(16, 8, dtype=b), torch.zeros(16, 8, dtype=b), torch.zeros(8, 16, dtype=b))
    for args in ((gate.float(), up, down), (gate, up[:8], down), (gate, up, down.T), (gate, up, gate), (gate[0], up, down)):
        with pytest.raises(fb.FlintMoeError):
            fb.flint_ffn_init(*args)
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    for m, out, co in ((torch.zeros(4, 6, dtype=f), torch.zeros(4, 6, dtype=f), STEPS), (torch.zeros(4, 6, dtype=f), torch.zeros(6, 4, dtype=b), STEPS),
                       (torch.zeros(6, 4, dtype=f).T, torch.zeros(4, 6, dtype=b), STEPS), (torch.zeros(6, dtype=f), torch.zeros(6, dtype=b), STEPS),
                       (torch.zeros(4, 6, dtype=torch.float16), torch.zeros(4, 6, dtype=b), STEPS),
                       (torch.zeros(4, 6, dtype=f), torch.zeros(4, 6, dtype=b), ((1.0, 2.0),))):
        with pytest.raises(fb.FlintMoeError):
            fb.flint_orthogonalize(m, out, co, 1e-7, ws)

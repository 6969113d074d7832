"""The fine-tuning operators without a GPU: host-side refusals, workspace sizes, and the float64 definitions
pinned to torch's automatic differentiation and to brute force."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import balance as ob
from oracle import lora as olora
from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _finetune import Pool, f64, router


@pytest.fixture(scope="module")
def lib():
    build()
    return fb.lib()


def handle(K=256, N=512, R=16, n=4, a=0x100000, b=0x200000, scale=0x300000):
    lora = fb.flint_lora()
    st = fb.lib().flint_lora_init(K, N, R, n, a, b, scale, ctypes.byref(lora))
    return st, lora


def test_lora_init_checks(lib):
    assert handle()[0] == fb.OK
    for kw in (dict(K=0), dict(K=12), dict(N=4), dict(N=70000), dict(R=0), dict(R=12), dict(R=136), dict(n=0), dict(n=1025)):
        assert handle(**kw)[0] == fb.EUNSUPPORTED, kw
    assert handle(a=None)[0] == fb.EINVAL and handle(scale=None)[0] == fb.EINVAL
    assert handle(a=0x100008)[0] == fb.EALIGN and handle(b=0x200002)[0] == fb.EALIGN and handle(scale=0x300002)[0] == fb.EALIGN
    assert lib.flint_lora_init(8, 8, 8, 1, 0x100000, 0x200000, 0x300000, None) == fb.EINVAL


def test_lora_workspaces(lib):
    _, l = handle()
    for f, most in ((fb.flint_lora_workspace_bytes, 65536), (fb.flint_lora_backward_workspace_bytes, 65536),
                    (fb.flint_gemv_lora_workspace_bytes, 32)):
        assert f(l, 0) == 0 and f(l, -1) == 0 and f(l, most + 1) == 0
        sizes = [f(l, t) for t in range(1, min(most, 300))] + [f(l, most)]
        assert all(0 < a <= b for a, b in zip(sizes, sizes[1:]))  # a workspace serves every smaller call
    l.rank = 12
    assert fb.flint_lora_workspace_bytes(l, 4) == 0


def test_lora_apply_refusals(lib):
    _, l = handle()
    ws = 0x4000000
    def call(x=0x1000000, ldx=256, ad=0x500000, T=40, yi=0x2000000, yo=0x3000000, ldy=512, w=ws, nb=1 << 30, lora=l):
        return lib.flint_lora_apply(None if lora is None else ctypes.byref(lora), x, ldx, ad, T, yi, yo, ldy, w, nb, None)
    assert call(T=0) == fb.OK and call(T=0, x=None, yo=None, w=None) == fb.OK
    assert call(lora=None) == fb.EINVAL
    for kw in (dict(T=-1), dict(T=65537), dict(x=None), dict(ad=None), dict(yo=None), dict(w=None), dict(ldx=248),
               dict(ldy=504), dict(nb=16), dict(yo=0x1000000), dict(yo=0x1000000 + 16), dict(yo=0x2000000 + 16),
               dict(yi=0x3000000 + 40 * 1024 - 16), dict(ldx=1 << 31), dict(ldy=1 << 31)):
        assert call(**kw) == fb.EINVAL, kw
    for kw in (dict(x=0x1000002), dict(yi=0x2000008), dict(yo=0x3000004), dict(ad=0x500002), dict(w=ws + 16), dict(ldx=260),
               dict(ldy=513)):
        assert call(**kw) == fb.EALIGN, kw


def test_row_strides_of_tensors(lib):
    """The binding reads row strides off the tensors, and refuses those that one stride cannot describe."""
    _, l = handle()  # K 256, N 512
    x, y = torch.zeros(40, 256, dtype=torch.bfloat16), torch.zeros(40, 1024, dtype=torch.bfloat16)
    def refused(f):
        with pytest.raises(fb.FlintMoeError) as e:
            f()
        assert e.value.status == fb.EINVAL
    go = lambda x, yi, yo: fb.flint_lora_apply(l, x, 0x500000, 40, yi, yo, 0x4000000, workspace_bytes=16, stream=0)  # noqa: E731
    refused(lambda: go(x, y[:, :512].contiguous(), y[:, 512:]))
    refused(lambda: go(x, y[:, :512], y[:, ::2]))
    refused(lambda: go(torch.zeros(256, 40, dtype=torch.bfloat16).t(), y[:, :512], y[:, :512]))
    assert fb._ld(x[:, :128], 40, 128, None) == 256 and fb._ld(x[:1, :128], 1, 128, None) == 128
    assert fb._ld(y, 40, 1024, None, y.clone()) == 1024 and fb._ld(y, 40, 1024, 7, x) == 7
    refused(lambda: fb.flint_lora_backward(l, x, 0x600000, 0x500000, 40, x, y[:, :256], 0x700000, 0x800000, 0x4000000,
                                           workspace_bytes=16, stream=0))


def test_gemv_lora_refusals(lib):
    _, l = handle(K=2048, N=2048)
    def call(N=2048, K=2048, fmt=fb.NVFP4, x=0x1000000, B=4, y=0x2000000, ad=0x500000, w=0x4000000, nb=1 << 30, p=0x6000000, st=None):
        return lib.flint_gemv_lora(p, N, K, fmt, x, B, y, ctypes.byref(l), ad, w, nb, st, None)
    assert call(B=0) == fb.OK
    assert call(N=2040) == fb.EUNSUPPORTED and call(fmt=2) == fb.EUNSUPPORTED
    for kw in (dict(B=33), dict(B=-1), dict(N=1024), dict(K=1024), dict(x=None), dict(y=None), dict(ad=None), dict(w=None),
               dict(p=None), dict(nb=100), dict(y=0x1000000)):
        assert call(**kw) == fb.EINVAL, kw
    for kw in (dict(x=0x1000008), dict(y=0x2000008), dict(ad=0x500001), dict(w=0x4000010), dict(p=0x6000004), dict(st=0x700002)):
        assert call(**kw) == fb.EALIGN, kw


def test_lora_backward_refusals(lib):
    _, l = handle()
    def call(x=0x1000000, ldx=256, dy=0x2000000, lddy=512, ad=0x500000, T=40, di=None, do=0x3000000, lddx=256, da=0x7000000,
             db=0x8000000, w=0x4000000, nb=1 << 30):
        return lib.flint_lora_backward(ctypes.byref(l), x, ldx, dy, lddy, ad, T, di, do, lddx, da, db, w, nb, None)
    for kw in (dict(T=-1), dict(T=65537), dict(x=None), dict(dy=None), dict(ad=None), dict(da=None), dict(db=None), dict(w=None),
               dict(nb=64), dict(ldx=128), dict(lddy=256), dict(lddx=8), dict(do=0x1000000), dict(do=0x2000010), dict(di=0x3000010),
               dict(da=0x100000), dict(db=0x200010), dict(db=0x100000), dict(da=0x1000000), dict(db=0x2000000), dict(da=0x3000000),
               dict(da=0x8000000 - 16), dict(ldx=1 << 31), dict(lddy=1 << 31), dict(lddx=1 << 31)):
        assert call(**kw) == fb.EINVAL, kw
    for kw in (dict(x=0x1000004), dict(dy=0x2000004), dict(do=0x3000004), dict(di=0x3000004), dict(da=0x7000002), dict(db=0x8000008),
               dict(w=0x4000020), dict(ad=0x500002), dict(ldx=260), dict(lddx=260)):
        assert call(**kw) == fb.EALIGN, kw


def test_balance_refusals(lib):
    cfg = fb.make_config()
    def call(z=0x1000000, idx=0x2000000, T=64, seq=0x3000000, n=2, alpha=0.1, loss=0x4000000, c=0x4100000, sc=0x4200000, st=0x4300000,
             w=0x4400000, nb=1 << 30, cfg=cfg):
        return lib.flint_moe_balance(ctypes.byref(cfg), z, idx, T, seq, n, ctypes.c_float(alpha), loss, c, sc, st, w, nb, None)
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(z=None), dict(idx=None), dict(n=0), dict(n=65537), dict(seq=None),
               dict(alpha=float("nan")), dict(alpha=float("inf")), dict(loss=None), dict(c=None), dict(sc=None), dict(st=None),
               dict(w=None), dict(nb=8)):
        assert call(**kw) == fb.EINVAL, kw
    for kw in (dict(z=0x1000004), dict(idx=0x2000002), dict(seq=0x3000001), dict(loss=0x4000002), dict(c=0x4100002), dict(w=0x4400004)):
        assert call(**kw) == fb.EALIGN, kw
    assert call(cfg=fb.make_config(top_k=17)) == fb.EUNSUPPORTED
    assert fb.flint_moe_balance_workspace_bytes(cfg, 0, 1) == 0 and fb.flint_moe_balance_workspace_bytes(cfg, 1, 0) == 0
    assert fb.flint_moe_balance_workspace_bytes(cfg, 1 << 20, 65536) > 0
    def back(z=0x1000000, idx=0x2000000, T=64, seq=0x3000000, n=2, sc=0x4200000, st=0x4300000, dl=None, dw=None, dz=0x5000000):
        return lib.flint_moe_balance_backward(ctypes.byref(cfg), z, idx, T, seq, n, ctypes.c_float(0.1), sc, st, dl, dw, dz, None)
    assert back(T=0) == fb.OK
    for kw in (dict(T=-1), dict(n=0), dict(seq=None), dict(z=None), dict(idx=None), dict(sc=None), dict(st=None), dict(dz=None),
               dict(dz=0x1000000), dict(dz=0x1000000 + 1024)):
        assert back(**kw) == fb.EINVAL, kw
    for kw in (dict(z=0x1000008), dict(dz=0x5000004), dict(dl=0x6000002), dict(dw=0x6000002)):
        assert back(**kw) == fb.EALIGN, kw


def test_lora_definition_against_autograd():
    p = Pool(40, 24, 32, 8, 3, 2)
    x, A, B, s = p.f64()
    a = p.adapter.numpy()
    tx, tA, tB = (torch.tensor(v, requires_grad=True) for v in (x, A, B))
    live = torch.tensor(p.live())
    ai = torch.tensor(np.where(p.live(), a, 0)).long()
    d = torch.einsum("tnr,trk,tk->tn", tB[ai], tA[ai], tx) * torch.tensor(s)[ai][:, None] * live[:, None]
    y = torch.tensor(f64(p.y)) + d
    assert np.allclose(olora.apply(x, a, A, B, s, f64(p.y)), y.detach().numpy(), rtol=1e-12, atol=1e-12)
    y.backward(torch.tensor(f64(p.dy)))
    dx, dA, dB = olora.backward(x, f64(p.dy), a, A, B, s, np.zeros_like(x))
    for got, want in ((dx, tx.grad), (dA, tA.grad), (dB, tB.grad)):
        assert np.allclose(got, want.numpy(), rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("renorm,scale", [(True, 1.0), (False, 2.0)])
def test_balance_definition_against_autograd(renorm, scale):
    T, E, k, at = 30, 12, 3, [0, 11, 11, 28]
    z, idx, start, dw = router(T, E, k, 4, at, pad=[5])
    zt = z.double().requires_grad_()
    s = torch.sigmoid(zt)
    c, tok = ob.counts(idx.numpy(), at, E)
    assert tok.tolist() == [10, 0, 17] and c.sum() == 27 * k
    total = torch.zeros((), dtype=torch.float64)
    for b in range(3):
        rows = [t for t in range(at[b], at[b + 1]) if idx[t, 0] >= 0]
        if rows:
            f = torch.tensor(c[b] * E / (k * len(rows)))
            total = total + 0.3 / 3 * (f * (s[rows] / s[rows].sum(1, keepdim=True)).mean(0)).sum()
    assert abs(float(total.detach()) - ob.loss(f64(z), idx.numpy(), at, k, 0.3)) < 1e-14
    rows = [t for t in range(at[0], at[-1]) if idx[t, 0] >= 0]
    w = torch.gather(s[rows], 1, idx[rows].long())
    w = scale * (w / w.sum(1, keepdim=True) if renorm else w)
    (1.25 * total + (w * dw[rows].double()).sum()).backward()
    got = ob.backward(f64(z), idx.numpy(), at, k, 0.3, 1.25, f64(dw), renorm, scale)
    assert np.allclose(got[:28], zt.grad.numpy()[:28], rtol=1e-10, atol=1e-15) and np.isnan(got[28:]).all()

"""The binding's own checks of the dense block's and the updates' tensors, without a GPU: types, shapes and strides that
the C ABI cannot see. A call that passes them reaches the library, which is a recorder here."""
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb

B16, F32 = torch.bfloat16, torch.float32
WS = dict(workspace_bytes=1 << 30, stream=0)


@pytest.fixture
def reached(monkeypatch):
    """The calls that reached the library."""
    calls = []

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return lambda *a: 4096
            return lambda *a: calls.append(name) or fb.OK

    monkeypatch.setattr(fb, "lib", Lib)
    fb._glu_packed_bytes.cache_clear()
    yield calls
    fb._glu_packed_bytes.cache_clear()


def refused(calls, f, *a, **kw):
    n = len(calls)
    with pytest.raises(fb.FlintMoeError) as e:
        f(*a, **kw)
    assert e.value.status == fb.EINVAL and len(calls) == n


def taken(calls, f, *a, **kw):
    n = len(calls)
    f(*a, **kw)
    assert len(calls) == n + 1


def bf(*s):
    return torch.zeros(*s, dtype=B16)


def test_gemv_glu(reached):
    I, K, B = 64, 256, 5
    good = dict(packed=torch.zeros(4096, dtype=torch.uint8), x=bf(B, K), h=bf(B, I), norm_weight=bf(K), dev_status=torch.zeros(1, dtype=torch.int32))

    def call(kw):
        v = {**good, **kw}
        fb.flint_gemv_glu(v["packed"], I, K, fb.NVFP4, v["x"], B, v["h"], v["norm_weight"], 1e-6, v["dev_status"], stream=0)

    for kw in ({}, dict(norm_weight=None, dev_status=None), dict(x=bf(B + 3, K), h=bf(B + 1, I)), dict(x=bf(B, K).view(torch.int16)),
               dict(x=bf(B, 4, K // 4), h=bf(B * I)), dict(x=bf(1, B, K), h=bf(1, B, I)), dict(packed=0x1000, x=0x2000, h=0x3000, norm_weight=0x4000, dev_status=0x5000)):
        taken(reached, call, kw)
    for kw in (dict(x=bf(B, K).float()), dict(x=bf(B, K).half()), dict(x=bf(B - 1, K)), dict(x=bf(B, K - 16)), dict(x=bf(B, 2 * K)),
               dict(x=bf(B, 2 * K)[:, :K]), dict(x=bf(2 * B, K)[::2]), dict(x=bf(K, B).T), dict(h=bf(B, I).float()), dict(h=bf(B - 1, I)), dict(h=bf(B, I // 2)),
               dict(h=bf(B, 2 * I)), dict(h=bf(B, 2 * I)[:, I:]), dict(norm_weight=bf(K // 2)), dict(norm_weight=torch.zeros(K)), dict(norm_weight=bf(2 * K)[::2]),
               dict(packed=torch.zeros(4095, dtype=torch.uint8)), dict(packed=torch.zeros(8192, dtype=torch.uint8)[::2]),
               dict(dev_status=torch.zeros(1)), dict(dev_status=torch.zeros(0, dtype=torch.int32))):
        refused(reached, call, kw)
    taken(reached, fb.flint_gemv_glu, torch.zeros(0, dtype=torch.uint8), I, K, fb.NVFP4, bf(0, K), 0, bf(0, I), stream=0)


def test_gemv_glu_pack(reached):
    I, K = 64, 256
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    good = {"codes": u8(I, K // 2), "scales": u8(I, K // 16), "global": torch.ones(1)}
    dst = u8(4096)
    for src in (good, {k: v.flatten() for k, v in good.items()}, {"codes": 0x1000, "scales": 0x2000, "global": 0x3000}, {**good, "global": torch.ones(())}):
        taken(reached, fb.flint_gemv_glu_pack, good, src, I, K, fb.NVFP4, dst, stream=0)
        taken(reached, fb.flint_gemv_glu_pack, src, good, I, K, fb.NVFP4, dst, stream=0)
    for kw in (dict(codes=u8(I, K)), dict(codes=u8(K // 2, I)), dict(codes=u8(I, K // 2).float()), dict(codes=u8(K // 2, I).T), dict(codes=u8(I * K // 2 - 1)),
               dict(scales=u8(I, K // 8)), dict(scales=u8(K // 16, I)), dict(scales=u8(I, K // 8)[:, ::2]), {"global": torch.ones(1, dtype=torch.float64)},
               {"global": torch.ones(2)}, {"global": torch.ones(0)}):
        for pair in (({**good, **kw}, good), (good, {**good, **kw})):
            refused(reached, fb.flint_gemv_glu_pack, *pair, I, K, fb.NVFP4, dst, stream=0)
    for ok in (bf(I, K), bf(I, K).view(torch.int16), bf(I * K)):
        taken(reached, fb.flint_gemv_glu_pack, {"bf16": ok}, {"bf16": bf(I, K)}, I, K, fb.BF16, dst, stream=0)
    for bad in (bf(K, I), bf(I, K).half(), bf(I, K).float(), bf(I, 2 * K)[:, :K], bf(K, I).T, bf(I - 8, K), bf(I * K + 1)):
        refused(reached, fb.flint_gemv_glu_pack, {"bf16": bf(I, K)}, {"bf16": bad}, I, K, fb.BF16, dst, stream=0)
        refused(reached, fb.flint_gemv_glu_pack, {"bf16": bad}, {"bf16": bf(I, K)}, I, K, fb.BF16, dst, stream=0)
    refused(reached, fb.flint_gemv_glu_pack, good, good, I, K, fb.NVFP4, u8(8192)[::2], stream=0)
    refused(reached, fb.flint_gemv_glu_pack, good, good, I, K, fb.NVFP4, dst, torch.zeros(1, dtype=torch.int64), stream=0)


def test_ffn_rows(reached):
    """Token rows of other types: their bits would be read as bf16."""
    T, H, I = 6, 64, 128
    f = fb.flint_ffn(H, I, 0x1000, 0x2000, 0x3000)
    ws = 0x100000
    rows, act = bf(T, H), bf(T, I)
    taken(reached, fb.flint_ffn_forward, f, rows, T, rows.clone(), ws, act, act.clone(), **WS)
    taken(reached, fb.flint_ffn_forward, f, rows.view(torch.int16), T, rows.view(torch.int16), ws, **WS)
    taken(reached, fb.flint_ffn_forward, f, 0x10000, T, 0x20000, ws, **WS)
    for bad in (rows.float(), rows.half(), rows.double(), torch.zeros(T, H, dtype=torch.int32), torch.zeros(T, 2 * H, dtype=torch.uint8)):
        refused(reached, fb.flint_ffn_forward, f, bad, T, rows, ws, **WS)
        refused(reached, fb.flint_ffn_forward, f, rows, T, bad, ws, **WS)
        refused(reached, fb.flint_ffn_forward, f, bad, T, rows, ws, ldx=H, **WS)
    w = [bf(I, H), bf(I, H), bf(H, I)]
    taken(reached, fb.flint_ffn_backward, f, rows, act, act, rows, T, rows, *w, ws, **WS)
    taken(reached, fb.flint_ffn_backward, f, rows, act, act, rows, T, None, *w, ws, **WS)
    for bad in (rows.float(), rows.half(), torch.zeros(T, H, dtype=torch.int32)):
        refused(reached, fb.flint_ffn_backward, f, bad, act, act, rows, T, rows, *w, ws, **WS)
        refused(reached, fb.flint_ffn_backward, f, rows, act, act, bad, T, rows, *w, ws, **WS)
        refused(reached, fb.flint_ffn_backward, f, rows, act, act, rows, T, bad, *w, ws, **WS)


def test_coefficients_are_triples(reached):
    """Steps of other lengths whose values add up to triples all the same."""
    m, out = torch.zeros(8, 16), bf(8, 16)
    taken(reached, fb.flint_orthogonalize, m, out, ((1.0, -0.5, 0.1), (1.0, 0.0, 0.0)), 1e-7, 0x1000, **WS)
    for bad in (((1.0, -0.5), (0.1, 1.0, 0.0, 0.0)), ((1.0, -0.5, 0.1, 0.0), (1.0, 0.0)), ((1.0,) * 6, ())):
        refused(reached, fb.flint_orthogonalize, m, out, bad, 1e-7, 0x1000, **WS)

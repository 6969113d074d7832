"""Low-rank adapters beside a projection (through the C ABI) against the float64
definition, with the bounds of _finetune (derived there).
"""
import numpy as np
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300 import layers
from w4a16_moe_decode_gb300.build import build

from _finetune import SLACK, SUM, Pool, check, f64
from oracle import moe, nvfp4
import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def ws_of(nbytes):
    # filled with NaN patterns: nothing may depend on what a workspace holds
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)


def apply(p, y_in, y_out=None, **kw):
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    y = torch.full((p.T, p.N), float("nan"), dtype=torch.bfloat16, device=DEV) if y_out is None else y_out
    fb.flint_lora_apply(lora, p.d_x, p.d_adapter, p.T, y_in, y, ws_of(fb.flint_lora_workspace_bytes(lora, p.T)), **kw)
    return y


def backward(p, dx_in, dx_out="new"):
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    if isinstance(dx_out, str):
        dx_out = torch.full((p.T, p.K), float("nan"), dtype=torch.bfloat16, device=DEV)
    dA, dB = (torch.full_like(v, float("nan")) for v in (p.d_A, p.d_B))
    fb.flint_lora_backward(lora, p.d_x, p.d_dy, p.d_adapter, p.T, dx_in, dx_out, dA, dB,
                           ws_of(fb.flint_lora_backward_workspace_bytes(lora, p.T)))
    return dx_out, dA, dB


# T, K, N, R, n: single tokens, the 32/33 border, tiles of 128 tokens and their borders, ranks that are no
# multiple of 16, widths that are no multiple of 64, one adapter, more adapters than tokens
SHAPES = [(1, 256, 256, 16, 1), (1, 8, 8, 8, 3), (2, 2048, 48, 128, 5), (7, 72, 200, 24, 4), (8, 512, 2048, 16, 2),
          (9, 2048, 520, 64, 1), (32, 256, 1000, 40, 40), (33, 1000, 256, 8, 3), (127, 64, 136, 16, 1), (128, 136, 64, 32, 1),
          (129, 256, 320, 64, 1), (300, 200, 1032, 56, 7), (1000, 328, 264, 128, 4), (2500, 72, 88, 8, 17)]


@pytest.mark.parametrize("T,K,N,R,n", SHAPES)
def test_apply(T, K, N, R, n):
    p = Pool(T, K, N, R, n, 11 * T + R).to(DEV)
    ref, tol = p.expect_apply(f64(p.y))
    y = apply(p, p.d_y)
    check(y, ref, tol, "apply")
    none = ~p.live()
    assert torch.equal(y.cpu()[none], p.y[none])  # no adapter: the base row, bit for bit
    assert torch.equal(apply(p, p.d_y), y)          # the same bits again
    inplace = p.d_y.clone()
    assert apply(p, inplace, inplace) is inplace and torch.equal(inplace, y)


@pytest.mark.parametrize("T,K,N,R,n", SHAPES)
def test_backward(T, K, N, R, n):
    p = Pool(T, K, N, R, n, 13 * T + R).to(DEV)
    refs, tols = p.expect_backward()
    got = backward(p, p.d_dx)
    for v, ref, tol, label in zip(got, refs, tols, ("dx", "dA", "dB")):
        check(v, ref, tol, label)
    assert torch.equal(got[0].cpu()[~p.live()], p.dx[~p.live()])
    again = backward(p, p.d_dx)
    assert all(torch.equal(u, v) for u, v in zip(got, again))
    _, dA, dB = backward(p, None, None)  # without dx
    assert torch.equal(dA, got[1]) and torch.equal(dB, got[2])


@pytest.mark.parametrize("T,K,N,R,n,run", [(700, 264, 328, 16, 3, 233), (1500, 72, 1000, 80, 2, 700), (640, 128, 40, 8, 5, 32),
                                           (520, 200, 96, 64, 4, 47), (300, 64, 264, 24, 2, 16)])
def test_runs_of_neighbouring_tokens(T, K, N, R, n, run):
    """Requests of `run` tokens each, so that tiles hold whole runs, parts of several and ragged ends: rows that move
    in boxes beside rows that are gathered."""
    p = Pool(T, K, N, R, n, 17 * T, [(t // run) % (n + 1) - 1 for t in range(T)]).to(DEV)
    check(apply(p, p.d_y), *p.expect_apply(f64(p.y)), "runs")
    inplace = p.d_y.clone()
    assert torch.equal(apply(p, inplace, inplace), apply(p, p.d_y))
    refs, tols = p.expect_backward()
    for v, ref, tol, label in zip(backward(p, p.d_dx), refs, tols, ("dx", "dA", "dB")):
        check(v, ref, tol, label)


@pytest.mark.parametrize("T", [5, 200])
def test_no_base_means_zero(T):
    p = Pool(T, 256, 264, 16, 3, 3).to(DEV)
    check(apply(p, None), *p.expect_apply(np.zeros((T, 264))), "apply without a base")
    p.dx.zero_()
    refs, tols = p.expect_backward()
    check(backward(p, None)[0], refs[0], tols[0], "dx without a base")


@pytest.mark.parametrize("T", [3, 32, 40, 400])
@pytest.mark.parametrize("which", ["none", "beyond", "last", "runs"])
def test_adapter_indexes(T, which):
    n = 6
    adapter = {"none": [-1] * T, "beyond": [n + t % 3 if t % 2 else -1 - t for t in range(T)],
               "last": [n - 1] * T, "runs": [(t * n) // T for t in range(T)]}[which]
    p = Pool(T, 128, 192, 16, n, 5, adapter).to(DEV)
    check(apply(p, p.d_y), *p.expect_apply(f64(p.y)), which)
    refs, tols = p.expect_backward()
    got = backward(p, p.d_dx)
    for v, ref, tol in zip(got, refs, tols):
        check(v, ref, tol, which)
    used = set(a for a in adapter if 0 <= a < n)
    for a in set(range(n)) - used:  # adapters without tokens: zero gradients, written
        assert not got[1][a].any() and not got[2][a].any()


@pytest.mark.parametrize("T", [6, 150])
def test_rows_stand_alone(T):
    """NaN and infinity in one token's rows reach that token's outputs and its adapter's gradients only."""
    n, bad_none, bad = 3, 1, 4
    adapter = [t % n for t in range(T)]
    adapter[bad_none] = -1
    p = Pool(T, 128, 192, 24, n, 6, adapter)
    clean = Pool(T, 128, 192, 24, n, 6, adapter).to(DEV)
    p.x[bad_none] = float("nan")
    p.dy[bad_none] = float("inf")
    p.x[bad, 3] = float("inf")
    p.dy[bad, 5] = float("nan")
    p.to(DEV)
    keep = torch.arange(T) != bad
    y, y0 = apply(p, p.d_y).cpu(), apply(clean, clean.d_y).cpu()
    assert torch.equal(y[keep], y0[keep]) and not torch.isfinite(y[bad].float()).all()
    (dx, dA, dB), (dx0, dA0, dB0) = backward(p, p.d_dx), backward(clean, clean.d_dx)
    assert torch.equal(dx.cpu()[keep], dx0.cpu()[keep])
    others = [a for a in range(n) if a != adapter[bad]]
    assert torch.equal(dA[others], dA0[others]) and torch.equal(dB[others], dB0[others])


@pytest.mark.parametrize("T", [4, 32, 133])
def test_strided_rows_and_guards(T):
    """Rows inside wider buffers: columns beside them and rows behind them stay as they were."""
    K, N, R, n = 192, 264, 16, 4
    p = Pool(T, K, N, R, n, 8).to(DEV)
    wide = lambda v, pad: torch.nn.functional.pad(v, (8, pad, 0, 3), value=float("nan"))  # noqa: E731
    p.d_x = wide(p.d_x, 16)[:T, 8:8 + K]
    yb = wide(p.d_y, 32)
    want = yb.clone()
    out = yb[:T, 8:8 + N]
    apply(p, out, out)
    check(out, *p.expect_apply(f64(p.y)), "strided")
    want[:T, 8:8 + N] = out
    assert torch.equal(want.view(torch.int16), yb.view(torch.int16))
    p.d_dy = wide(p.d_dy, 24)[:T, 8:8 + N]
    db = wide(p.d_dx, 8)
    want = db.clone()
    dx = db[:T, 8:8 + K]
    refs, tols = p.expect_backward()
    got = backward(p, dx, dx)
    for v, ref, tol in zip(got, refs, tols):
        check(v, ref, tol, "strided backward")
    want[:T, 8:8 + K] = dx
    assert torch.equal(want.view(torch.int16), db.view(torch.int16))


@pytest.mark.parametrize("T", [20, 200])
def test_without_dx_its_arguments_are_not_read(T):
    p = Pool(T, 72, 136, 16, 3, 60 + T).to(DEV)
    _, dA0, dB0 = backward(p, None, None)
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    dA, dB = (torch.full_like(v, float("nan")) for v in (p.d_A, p.d_B))
    fb.flint_lora_backward(lora, p.d_x, p.d_dy, p.d_adapter, T, p.d_dx, None, dA, dB,
                           ws_of(fb.flint_lora_backward_workspace_bytes(lora, T)), lddx=0)
    assert torch.equal(dA, dA0) and torch.equal(dB, dB0)


def test_zero_tokens():
    p = Pool(0, 64, 64, 8, 2, 1).to(DEV)
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    fb.flint_lora_apply(lora, p.d_x, p.d_adapter, 0, None, p.d_y, torch.empty(0, dtype=torch.uint8, device=DEV))
    dA, dB = (torch.full_like(v, float("nan")) for v in (p.d_A, p.d_B))
    fb.flint_lora_backward(lora, None, None, None, 0, None, None, dA, dB, None, workspace_bytes=0)
    assert not dA.any() and not dB.any()


def test_long_batch_of_many_adapters():
    """More tokens and adapters than one plan block's first pass; checked on a sample of rows."""
    T, K, N, R, n = 20000, 64, 72, 8, 300
    p = Pool(T, K, N, R, n, 9).to(DEV)
    y = apply(p, p.d_y)
    rows = torch.randperm(T, generator=torch.Generator().manual_seed(1))[:400]
    q = Pool(T, K, N, R, n, 9)
    for k in ("x", "y", "adapter"):
        setattr(q, k, getattr(q, k)[rows])
    check(y.cpu()[rows], *q.expect_apply(f64(q.y)), "long batch")


def gemv_case(B, K, N, R, n, fmt, seed, adapter=None):
    p = Pool(B, K, N, R, n, seed, adapter).to(DEV)
    packed, canon = layers.synth_dense(N, K, seed, 0, fmt, DEV)
    w = synth.matrix_f32(seed, 0, synth.DOWN, 0, N, K, 0.02)
    m = moe.NVFP4Matrix(*nvfp4.quantize(w)) if fmt == fb.NVFP4 else moe.BF16Matrix(synth.f32_to_bf16_bits(w))
    W = np.float64(m.G) * m.c()
    return p, packed, W


def gemv_lora(p, packed, fmt, stream=None):
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    y = torch.full((p.T, p.N), float("nan"), dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    fb.flint_gemv_lora(packed, p.N, p.K, fmt, p.d_x, p.T, y, lora, p.d_adapter,
                       ws_of(fb.flint_gemv_lora_workspace_bytes(lora, p.T)), dev_status=status, stream=stream)
    assert int(status.item()) == 0
    return y


@pytest.mark.parametrize("B,K,N,R,n,fmt", [(1, 256, 64, 8, 1, fb.NVFP4), (1, 2048, 2048, 16, 4, fb.NVFP4),
                                           (5, 768, 1040, 72, 3, fb.BF16), (8, 4096, 272, 32, 8, fb.NVFP4),
                                           (17, 512, 256, 128, 30, fb.NVFP4), (32, 2048, 512, 64, 32, fb.BF16),
                                           (20, 256, 4352, 128, 2, fb.NVFP4), (9, 512, 8208, 40, 3, fb.NVFP4),
                                           (32, 8192, 64, 24, 2, fb.NVFP4)])
def test_gemv_lora(B, K, N, R, n, fmt):
    p, packed, W = gemv_case(B, K, N, R, n, fmt, 70 + B)
    x = f64(p.x)
    base = x @ W.T
    ref, tol = p.expect_apply(base)
    # the base's FP32 sum over K, and its f16 rows: x / max|x| is exact down to 2^-24 of its largest value
    tol = tol + SLACK * ((K + 4) * SUM * (np.abs(x) @ np.abs(W).T) + 2.0 ** -24 * np.abs(x).max(1)[:, None] * np.abs(W).sum(1)[None, :])
    y = gemv_lora(p, packed, fmt)
    check(y, ref, tol, "gemv_lora")
    assert torch.equal(gemv_lora(p, packed, fmt), y)
    # a batch without adapters is the plain GEMV
    p.d_adapter.fill_(-1)
    plain = torch.empty_like(y)
    fb.flint_gemv(packed, N, K, fmt, p.d_x, B, plain)
    assert torch.equal(gemv_lora(p, packed, fmt), plain)


def test_gemv_lora_follows_the_kernel_before_it():
    """x is the output of the GEMV before on the same stream, many times in a row: the adapters' kernels, which
    start early, must see the finished rows."""
    D, R, n, B = 2048, 16, 4, 3
    p, packed, W = gemv_case(B, D, D, R, n, fb.NVFP4, 90)
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    ws = ws_of(fb.flint_gemv_lora_workspace_bytes(lora, B))
    rows = [p.d_x] + [torch.empty_like(p.d_x) for _ in range(12)]
    for i in range(12):
        fb.flint_gemv_lora(packed, D, D, fb.NVFP4, rows[i], B, rows[i + 1], lora, p.d_adapter, ws)
    torch.cuda.synchronize()
    for i in range(12):  # each step alone
        y = torch.empty_like(p.d_x)
        fb.flint_gemv_lora(packed, D, D, fb.NVFP4, rows[i], B, y, lora, p.d_adapter, ws)
        torch.cuda.synchronize()
        assert torch.equal(y, rows[i + 1]), i


def test_streams_and_graphs():
    """Two calls at once on two streams with a workspace each, then a captured and replayed run of the three
    operators on new inputs."""
    ps = [Pool(T, 256, 264, 16, 5, 20 + T).to(DEV) for T in (20, 300)]
    want = [(apply(p, p.d_y), backward(p, p.d_dx)) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for p, s in zip(ps, streams):
        with torch.cuda.stream(s):
            got.append((apply(p, p.d_y), backward(p, p.d_dx)))
    torch.cuda.synchronize()
    for (y, g), (y0, g0) in zip(got, want):
        assert torch.equal(y, y0) and all(torch.equal(u, v) for u, v in zip(g, g0))
    p = ps[1]
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    ws = ws_of(max(fb.flint_lora_workspace_bytes(lora, p.T), fb.flint_lora_backward_workspace_bytes(lora, p.T)))
    y, dx, dA, dB = (torch.empty_like(v) for v in (p.d_y, p.d_dx, p.d_A, p.d_B))
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        fb.flint_lora_apply(lora, p.d_x, p.d_adapter, p.T, p.d_y, y, ws)
        fb.flint_lora_backward(lora, p.d_x, p.d_dy, p.d_adapter, p.T, p.d_dx, dx, dA, dB, ws)
    for seed in (1, 2):
        q = Pool(300, 256, 264, 16, 5, seed).to(DEV)
        for k in ("x", "y", "dy", "dx", "A", "B", "scale", "adapter"):
            getattr(p, "d_" + k).copy_(getattr(q, "d_" + k))
        g.replay()
        torch.cuda.synchronize()
        y0, g0 = apply(q, q.d_y), backward(q, q.d_dx)
        assert torch.equal(y, y0) and all(torch.equal(u, v) for u, v in zip((dx, dA, dB), g0))


def test_gemv_lora_in_a_graph_and_beside_another_stream():
    """Captured and replayed on new rows, indexes and adapters while the same operator runs on another stream with its
    own workspace."""
    D, R, n, B = 2048, 16, 6, 12
    p, packed, _ = gemv_case(B, D, D, R, n, fb.NVFP4, 95)
    q, _, _ = gemv_case(B, D, D, R, n, fb.NVFP4, 96)
    want_q = gemv_lora(q, packed, fb.NVFP4)
    lora = fb.flint_lora_init(p.d_A, p.d_B, p.d_scale)
    ws = ws_of(fb.flint_gemv_lora_workspace_bytes(lora, B))
    y = torch.empty_like(p.d_x)
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        fb.flint_gemv_lora(packed, D, D, fb.NVFP4, p.d_x, B, y, lora, p.d_adapter, ws)
    for seed in (1, 2):
        r = Pool(B, D, D, R, n, seed).to(DEV)
        for k in ("x", "A", "B", "scale", "adapter"):
            getattr(p, "d_" + k).copy_(getattr(r, "d_" + k))
        torch.cuda.synchronize()
        got_q = []
        with torch.cuda.stream(other):
            got_q.append(gemv_lora(q, packed, fb.NVFP4))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got_q[0], want_q) and torch.equal(y, gemv_lora(r, packed, fb.NVFP4))


@pytest.mark.parametrize("T,n", [(32, 1), (32, 3), (29, 29), (17, 2), (9, 1)])
@pytest.mark.parametrize("R", [8, 48, 128])
def test_groups_of_many_rows_of_one_adapter(T, n, R):
    """Up to 32 rows of one adapter: more than one tile of 8 tokens in a cluster, more pieces of B than are held."""
    p = Pool(T, 520, 4360, R, n, 100 * T + R, [t % n for t in range(T)]).to(DEV)
    check(apply(p, p.d_y), *p.expect_apply(f64(p.y)), "groups")


def test_gradients_against_differences():
    """The kernels' gradients along a random direction against central differences of the float64 definition of
    L = sum y dy."""
    from oracle import lora as olora
    p = Pool(150, 136, 200, 24, 3, 30).to(DEV)
    dx, dA, dB = (f64(v) for v in backward(p, p.d_dx))
    _, tols = p.expect_backward()
    x, A, B, s = p.f64()
    dy, a = f64(p.dy), p.adapter.numpy()
    rng = np.random.default_rng(0)
    vx, vA, vB = (rng.standard_normal(v.shape) for v in (x, A, B))
    L = lambda e: float((olora.apply(x + e * vx, a, A + e * vA, B + e * vB, s, np.zeros_like(dy)) * dy).sum())  # noqa: E731
    e = 1e-5
    num = (L(e) - L(-e)) / (2 * e)
    ana = float((vx * (dx - f64(p.dx))).sum() + (vA * dA).sum() + (vB * dB).sum())
    # the gradients' own bounds along the direction, and the differences' third-order term (L is cubic in e)
    bound = sum(float((t * np.abs(v)).sum()) for t, v in zip(tols, (vx, vA, vB)))
    third = abs(L(1.0) - L(-1.0)) / 2 + abs(num)
    size = float(np.abs(olora.apply(x, a, A, B, s, np.zeros_like(dy)) * dy).sum())  # its FP64 sums' rounding
    assert abs(ana - num) <= bound + e * e * third + 1e-14 * size / e

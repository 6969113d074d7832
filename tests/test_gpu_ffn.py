"""The dense gated block on BF16 weights and its gradients (through the C ABI) against the float64 definition, with the
bounds of _dense (derived there), and each error's norm below 2^-8 of the result's: two roundings to bf16, each of at
most 2^-8 / sqrt(3) in the root mean square, and FP32 sums beside them.
"""
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _dense import Block, near
from _finetune import check

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("dx", "dgate", "dup", "ddown")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def ws_of(nbytes):
    # filled with NaN patterns: nothing may depend on what a workspace holds
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)


def nans(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)


def handle(p):
    return fb.flint_ffn_init(p.d_gate, p.d_up, p.d_down)


def forward(p, save=True, **kw):
    f = handle(p)
    ws = ws_of(fb.flint_ffn_workspace_bytes(f, p.T))
    y, g, u = nans(p.T, p.H), nans(p.T, p.I) if save else None, nans(p.T, p.I) if save else None
    fb.flint_ffn_forward(f, p.d_x, p.T, y, ws, g, u, **kw)
    assert fb.flint_moe_read_status(ws) == (fb.OK, 0)
    return (y, g, u) if save else y


def backward(p, dx=True, weights=True):
    f = handle(p)
    ws = ws_of(fb.flint_ffn_backward_workspace_bytes(f, p.T))
    out = [nans(p.T, p.H) if dx else None] + [nans(*v.shape) if weights else None for v in (p.gate, p.up, p.down)]
    fb.flint_ffn_backward(f, p.d_x, p.d_g, p.d_u, p.d_dy, p.T, *out, ws)
    assert fb.flint_moe_read_status(ws) == (fb.OK, 0)
    return out


# T, H, I: single tokens, the smallest sizes, tiles of 128 and 256 and their borders, reductions that are no multiple of
# 64 or 16, long and short ones, widths that end inside a tile
SHAPES = [(1, 8, 8), (1, 2048, 512), (2, 72, 200), (7, 256, 64), (31, 136, 1032), (33, 1000, 40), (64, 64, 64), (127, 64, 136), (128, 256, 128),
          (129, 128, 264), (200, 520, 328), (256, 256, 256), (257, 264, 520), (513, 200, 776), (1000, 328, 72), (2050, 136, 96)]
# enough tiles of 256 x 256 for pairs of CTAs: in the first products, the last ones, and the weights' gradients
LARGE = [(1300, 72, 1704), (2600, 2040, 72), (40, 2040, 2600), (4100, 1288, 1160)]
# one tile a CTA and SM with long runs of k-blocks, in the second product and in the first
LONG = [(1024, 832, 2600), (100, 2600, 8000)]


@pytest.mark.parametrize("T,H,I", SHAPES + LARGE + LONG)
def test_forward(T, H, I):
    p = Block(T, H, I, 7 * T + H).to(DEV)
    refs, tols = p.expect_forward()
    got = forward(p)
    for v, ref, tol, label in zip(got, refs, tols, ("y", "g", "u")):
        check(v, ref, tol, label)
        near(v, ref, 2.0 ** -8, label)
    assert torch.equal(forward(p, save=False), got[0])
    assert torch.equal(forward(p)[0], got[0])  # the same bits again


@pytest.mark.parametrize("T,H,I", SHAPES + LARGE)
def test_backward(T, H, I):
    p = Block(T, H, I, 5 * T + I).to(DEV)
    refs, tols = p.expect_backward()
    got = backward(p)
    for v, ref, tol, label in zip(got, refs, tols, NAMES):
        check(v, ref, tol, label)
        near(v, ref, 2.0 ** -8, label)
    again = backward(p)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert torch.equal(backward(p, weights=False)[0], got[0])
    assert all(torch.equal(a, b) for a, b in zip(backward(p, dx=False)[1:], got[1:]))


def test_large_gate_values():
    """Gates of -24 .. 24 and beyond: sigmoids at both ends."""
    p = Block(150, 128, 192, 3, sigma=8.0).to(DEV)
    assert float(p.g.abs().max()) > 20
    p.g.clamp_(-24, 24)
    p.d_g = p.g.to(DEV)
    refs, tols = p.expect_backward()
    for v, ref, tol, label in zip(backward(p), refs, tols, NAMES):
        check(v, ref, tol, label)
    p.g[::3] = -300.0  # the sigmoid and everything behind it vanish
    p.g[1::3] = 300.0  # the sigmoid is one
    p.d_g = p.g.to(DEV)
    refs, tols = p.expect_backward()
    for v, ref, tol, label in zip(backward(p), refs, tols, NAMES):
        check(v, ref, tol, label)


def apart(v, ld, rows=None):
    """The rows of v, ld elements apart, in a buffer of NaN."""
    n, cols = v.shape
    out = nans((rows or n) * ld)[: (rows or n) * ld].view(rows or n, ld)
    out[:n, :cols] = v
    return out


@pytest.mark.parametrize("T", [3, 140])
def test_strides_and_rows_behind_the_last(T):
    p = Block(T, 136, 200, 5).to(DEV)
    y, g, u = forward(p)
    f = handle(p)
    x, yy = apart(p.d_x, 152, T + 5), nans(T + 5, 144)
    gg, uu = nans(T + 2, 200), nans(T + 2, 200)
    fb.flint_ffn_forward(f, x[:T, :136], T, yy[:T, :136], ws_of(fb.flint_ffn_workspace_bytes(f, T + 9)), gg[:T], uu[:T])
    assert torch.equal(yy[:T, :136], y) and torch.equal(gg[:T], g) and torch.equal(uu[:T], u)
    assert yy[T:].isnan().all() and yy[:, 136:].isnan().all() and gg[T:].isnan().all() and uu[T:].isnan().all()
    want = backward(p)
    dx, dy = nans(T + 5, 160), apart(p.d_dy, 144)
    dw = [torch.empty_like(v) for v in (p.d_gate, p.d_up, p.d_down)]
    fb.flint_ffn_backward(f, x[:T, :136], p.d_g, p.d_u, dy[:, :136], T, dx[:T, :136], *dw,
                          ws_of(fb.flint_ffn_backward_workspace_bytes(f, T)))
    assert torch.equal(dx[:T, :136], want[0]) and dx[T:].isnan().all() and dx[:, 136:].isnan().all()
    assert all(torch.equal(a, b) for a, b in zip(dw, want[1:]))


def test_rows_past_32_bits():
    T, ld = 150, 1 << 24
    assert (T - 1) * ld > 1 << 31
    p = Block(T, 72, 136, 6).to(DEV)
    y, g, u = forward(p)
    want = backward(p)
    big = [torch.empty((T - 1) * ld + 72, dtype=torch.bfloat16, device=DEV).as_strided((T, 72), (ld, 1)) for _ in range(2)]
    big[0].copy_(p.d_x)
    f = handle(p)
    fb.flint_ffn_forward(f, big[0], T, big[1], ws_of(fb.flint_ffn_workspace_bytes(f, T)))
    assert torch.equal(big[1], y)
    big[1].copy_(p.d_dy)
    dx = torch.empty((T - 1) * ld + 72, dtype=torch.bfloat16, device=DEV).as_strided((T, 72), (ld, 1))
    dw = [torch.empty_like(v) for v in (p.d_gate, p.d_up, p.d_down)]
    fb.flint_ffn_backward(f, big[0], p.d_g, p.d_u, big[1], T, dx, *dw, ws_of(fb.flint_ffn_backward_workspace_bytes(f, T)))
    assert torch.equal(dx, want[0]) and all(torch.equal(a, b) for a, b in zip(dw, want[1:]))
    del big, dx
    torch.cuda.empty_cache()


def test_no_tokens():
    p = Block(1, 64, 72, 8).to(DEV)
    f = handle(p)
    dw = [nans(*v.shape) for v in (p.gate, p.up, p.down)]
    none = torch.empty(0, 72, dtype=torch.bfloat16, device=DEV)
    fb.flint_ffn_backward(f, p.d_x, none, none, p.d_dy, 0, None, *dw, ws_of(256))
    assert all(not v.any() for v in dw)
    y = nans(1, 64)
    fb.flint_ffn_forward(f, p.d_x, 0, y, ws_of(256))
    assert y.isnan().all()


def test_streams_and_graphs():
    """Two calls at once on two streams, and a captured step replayed on other values."""
    ps = [Block(T, 264, 136, T).to(DEV) for T in (140, 300)]
    want = [(forward(p), backward(p)) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for p, s in zip(ps, streams):
        with torch.cuda.stream(s):
            got.append((forward(p), backward(p)))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(v, w) for v, w in zip((*a[0], *a[1]), (*b[0], *b[1])))
    p, q = ps[0], Block(140, 264, 136, 9).to(DEV)
    f = handle(p)
    y, g, u = nans(140, 264), nans(140, 136), nans(140, 136)
    out = [nans(140, 264)] + [torch.empty_like(v) for v in (p.d_gate, p.d_up, p.d_down)]
    ws = ws_of(fb.flint_ffn_backward_workspace_bytes(f, 140))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fb.flint_ffn_forward(f, p.d_x, 140, y, ws, g, u)
        fb.flint_ffn_backward(f, p.d_x, g, u, p.d_dy, 140, *out, ws)
    for k in ("x", "dy", "gate", "up", "down"):
        getattr(p, "d_" + k).copy_(getattr(q, "d_" + k))
    for _ in range(2):
        for v in (y, g, u, *out):
            v.fill_(float("nan"))
        graph.replay()
    fy, fg, fu = forward(q)
    q.d_g, q.d_u = fg, fu
    assert torch.equal(y, fy) and torch.equal(g, fg) and torch.equal(u, fu)
    assert all(torch.equal(a, b) for a, b in zip(out, backward(q)))

"""Calls of the dense block and of orthogonalised updates that run at the same time on two streams, each with a workspace
of its own: nothing is shared between them. All calls are issued behind work that keeps both streams busy, and nothing
waits for the device until the last is in its stream."""
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build

from _dense import STEPS, Block, momentum

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def ws_of(nbytes):
    return torch.full((nbytes,), 0xFF, dtype=torch.uint8, device=DEV)


class Step:
    """A block's forward and backward calls, with outputs and workspaces in hand."""

    def __init__(self, T, H, I, seed):
        p = self.p = Block(T, H, I, seed).to(DEV)
        self.f = fb.flint_ffn_init(p.d_gate, p.d_up, p.d_down)
        self.ws = [ws_of(fb.flint_ffn_workspace_bytes(self.f, T)), ws_of(fb.flint_ffn_backward_workspace_bytes(self.f, T))]
        self.outs = [torch.empty_like(v) for v in (p.d_x, p.d_g, p.d_u, p.d_x, p.d_gate, p.d_up, p.d_down)]

    def call(self, stream):
        p, (y, g, u, *grads) = self.p, self.outs
        fb.flint_ffn_forward(self.f, p.d_x, p.T, y, self.ws[0], g, u, stream=stream)
        fb.flint_ffn_backward(self.f, p.d_x, g, u, p.d_dy, p.T, *grads, self.ws[1], stream=stream)


class Update:
    def __init__(self, n, rows, cols, seed):
        self.m = momentum(n, rows, cols, seed, "noise").to(DEV)
        self.ws = [ws_of(fb.flint_orthogonalize_workspace_bytes(n, rows, cols))]
        self.outs = [torch.empty(n, rows, cols, dtype=torch.bfloat16, device=DEV)]

    def call(self, stream):
        fb.flint_orthogonalize(self.m, self.outs[0], STEPS, 1e-7, self.ws[0], stream=stream)


# Two of a kind and different ones side by side: clusters along K, one tile a CTA, pairs of CTAs; the cluster kernel of
# updates (of four, of eight), the products of one update, of a batch
PAIRS = [((Step, 77, 512, 1032, 1), (Step, 77, 512, 1032, 2)), ((Step, 40, 2040, 520, 1), (Step, 300, 264, 136, 2)),
         ((Step, 1300, 264, 2600, 1), (Step, 1300, 264, 2600, 2)), ((Step, 1300, 264, 2600, 1), (Step, 77, 512, 1032, 2)),
         ((Update, 6, 64, 2048, 1), (Update, 6, 64, 2048, 2)), ((Update, 4, 128, 2048, 1), (Update, 8, 16, 2048, 2)),
         ((Update, 1, 256, 1024, 1), (Update, 1, 256, 1024, 2)), ((Update, 76, 200, 264, 1), (Update, 3, 300, 260, 2)),
         ((Update, 16, 64, 2048, 1), (Step, 77, 512, 1032, 2)), ((Update, 20, 512, 512, 1), (Step, 1300, 264, 2600, 2))]


@pytest.mark.parametrize("one,other", PAIRS)
def test_two_streams(one, other):
    ops = [kind(*args) for kind, *args in (one, other)]
    want = []
    for op in ops:
        for v in op.outs:
            v.fill_(float("nan"))
        op.call(None)
        torch.cuda.synchronize()
        want.append([v.clone() for v in op.outs])
        assert not any(v.isnan().any() for v in want[-1])
    streams = [torch.cuda.Stream() for _ in ops]
    a = torch.randn(4096, 4096, device=DEV)
    rounds, kept = 6, [[], []]
    copies = [[[torch.empty_like(v) for v in op.outs] for _ in range(rounds)] for op in ops]
    torch.cuda.synchronize()
    busy = torch.cuda.Event()
    for _ in range(4):
        a = a @ a * 1e-3  # (a few milliseconds, in which the calls below are issued)
    busy.record()
    for s in streams:
        s.wait_event(busy)
    for r in range(rounds):
        for op, s, c, k in zip(ops, streams, copies, kept):
            op.call(s)
            with torch.cuda.stream(s):
                for v, w in zip(c[r], op.outs):
                    v.copy_(w)
                k.append(c[r])
    torch.cuda.synchronize()
    for op, k, w in zip(ops, kept, want):
        assert all(torch.equal(x, y) for c in k for x, y in zip(c, w))
        for ws in op.ws:
            assert fb.flint_moe_read_status(ws) == (fb.OK, 0)

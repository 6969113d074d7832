"""The binding's own checks of the fine-tuning operators' tensors, without a GPU: shapes, types and strides that the C
ABI cannot see."""
import pytest
import torch

from w4a16_moe_decode_gb300 import binding as fb
from w4a16_moe_decode_gb300.build import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    fb.lib()


def refused(f, *a, **kw):
    with pytest.raises(fb.FlintMoeError) as e:
        f(*a, **kw)
    assert e.value.status == fb.EINVAL


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def test_row_strides_of_batched_tensors():
    """Tokens of a [batch, sequence, width] view: the one stride that its rows share, or a refusal."""
    B, S, K = 3, 7, 64
    ld = lambda t, rows=B * S, like=None: fb._ld(t, rows, K, None, like)  # noqa: E731
    qkv = bf(B, S, 3 * K)
    assert ld(qkv[:, :, :K]) == ld(qkv[:, :, K:2 * K]) == ld(qkv.view(B, S, 3, K)[:, :, 1]) == 3 * K
    assert ld(bf(B, S, K)) == ld(bf(B, S, 4, K // 4)) == ld(bf(B, S, 1, K)) == ld(bf(B * S * K)) == K
    assert ld(qkv.view(B, S, 3, 4, K // 4)[:, :, 2]) == 3 * K
    assert ld(bf(B, 2 * S, K)[:, ::2]) == 2 * K                                # every other token of all sequences
    assert ld(qkv[1:2, :, :K], S) == 3 * K and ld(qkv[:, 2:3, :K], B) == 3 * K * S
    assert ld(qkv[2:, 3:4, :K], 1) == K
    refused(ld, bf(B, S + 1, K)[:, :S])                                        # sequences cut short: two strides
    refused(ld, bf(S, B, K).transpose(0, 1))
    refused(ld, bf(B, K, S).transpose(1, 2))
    refused(ld, bf(B, S, 2 * K)[:, :, ::2])
    refused(ld, bf(B, S, 2 * K))                                               # whole rows of another width
    refused(ld, bf(B, S, 4, K // 2)[:, :, :2].transpose(2, 3))
    refused(ld, bf(1, 1, 2 * K)[:, :, ::2], 1)
    refused(ld, bf(2 * B * S * K)[::2])
    refused(ld, bf(B * S - 1, K))                                              # fewer rows or columns than are read
    refused(ld, bf(B * S, K - 8))
    refused(ld, bf(B, S - 1, K))
    refused(ld, bf(B * S * K - 1))
    assert ld(bf(B, S, K), like=qkv.view(B * S, 3 * K)[:, :K].contiguous()) == K
    refused(ld, bf(B, S, K), like=qkv[:, :, :K])
    refused(ld, qkv[:, :, :K], like=bf(B, S, K))
    refused(ld, bf(B, S, K), like=bf(B, S + 1, K)[:, :S])


def test_calls_refuse_such_rows(monkeypatch):
    """Before anything reaches the library."""
    lora = fb.flint_lora_init(0x100000, 0x200000, 0x300000, 64, 64, 16, 4)
    wide, flat = bf(2, 9, 64)[:, :8], bf(2, 8, 64)

    def reached():
        raise AssertionError("the library was called")

    monkeypatch.setattr(fb, "lib", lambda: type("L", (), {"__getattr__": lambda self, name: lambda *a: reached()})())
    ad, ws, kw = 0x500000, 0x4000000, dict(workspace_bytes=1 << 30, stream=0)
    for x, yi, yo in ((wide, flat, flat), (flat, wide, flat), (flat, None, wide)):
        refused(fb.flint_lora_apply, lora, x, ad, 16, yi, yo, ws, **kw)
    for x, dy, di, do in ((wide, flat, None, None), (flat, wide, None, None), (flat, flat, wide, flat), (flat, flat, None, wide)):
        refused(fb.flint_lora_backward, lora, x, dy, ad, 16, di, do, 0x700000, 0x800000, ws, **kw)


def test_pools_of_adapters():
    n, R, K, N = 4, 16, 64, 128
    a, b, s = bf(n, R, K), bf(n, N, R), torch.zeros(n)
    lora = fb.flint_lora_init(a, b, s)
    assert (lora.num_adapters, lora.rank, lora.in_dim, lora.out_dim) == (n, R, K, N)
    fb.flint_lora_init(a.view(torch.int16), b.view(torch.int16), s)              # the values' bits
    fb.flint_lora_init(a.flatten(), b.flatten(), s, K, N, R, n)
    fb.flint_lora_init(a, b, s, K, N, R, n - 1)                                 # the first of a pool
    fb.flint_lora_init(0x100000, 0x200000, 0x300000, K, N, R, n)
    for bad in (bf(n, N, R // 2), bf(n, N, 2 * R), bf(n - 1, N, R), bf(n + 1, N, R), bf(n, R, N).transpose(1, 2), bf(n, N, 2 * R)[:, :, :R],
                torch.zeros(n, N, R), torch.zeros(n, N, R, dtype=torch.float16), bf(n, N * R)):
        refused(fb.flint_lora_init, a, bad, s)
    for bad in (bf(n, K, R).transpose(1, 2), bf(n, R, 2 * K)[:, :, :K], torch.zeros(n, R, K), bf(n * R, K), bf(2 * n, R, K)[::2]):
        refused(fb.flint_lora_init, bad, b, s)
    for bad in (torch.zeros(n - 1), torch.zeros(n, dtype=torch.float64), bf(n), torch.zeros(2 * n)[::2]):
        refused(fb.flint_lora_init, a, b, bad)
    refused(fb.flint_lora_init, a, b, s, K, N, R, n + 1)                        # past the tensors' ends
    refused(fb.flint_lora_init, a, b, s, 2 * K, N, R, n)

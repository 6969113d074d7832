"""Measured cases of the fine-tuning operators: low-rank adapters beside a shared projection (serving and
training) and the router's balance loss with its gradient.

Each case is one call a program makes:
  gemv_lora         y = W x + scale_a B_a (A_a x) for up to 32 rows on a packed NVFP4 or BF16 matrix W
  lora              y = y_in + scale_a B_a (A_a x) for many tokens of many requests (the projection is y_in)
  lora_backward     dx, dA and dB of the same from dy
  balance           balance loss, per-expert counts (total and per sequence) from router logits and picks
  balance_backward  the logits' gradient, of the loss and (with dw) of the routing weights

`run` computes them from elementary torch operations in 32 bits, or, where `own` is true, by the library.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoding request with an adapter on a hidden-sized projection: latency
        dict(name="gemv_lora 1x2048x2048 r16", op="gemv_lora", T=1, K=2048, N=2048, R=16, n=8, none=0, fmt="nvfp4"),
        # a decode batch of 13 requests, three of them on the base model, on the dense down projection
        dict(name="gemv_lora 13x8192x2048 r32", op="gemv_lora", T=13, K=8192, N=2048, R=32, n=16, none=3, fmt="nvfp4"),
        # the largest decode batch, each row another request's adapter, wide projection
        dict(name="gemv_lora 32x2048x8192 r64", op="gemv_lora", T=32, K=2048, N=8192, R=64, n=40, none=0, fmt="nvfp4"),
        # a step that mixes the rows of 40 requests (chunked prompts and single tokens), odd sizes
        dict(name="lora 777x1000x2040 r8", op="lora", T=777, K=1000, N=2040, R=8, n=24, reqs=40, none=3, mixed=True),
        # prompts of 21 requests on a hidden-sized projection
        dict(name="lora 4096x2048x2048 r16", op="lora", T=4096, K=2048, N=2048, R=16, n=16, reqs=21, none=2, mixed=False),
        # a full prefill step, few adapters of a high rank, wide projection
        dict(name="lora 8192x2048x8192 r64", op="lora", T=8192, K=2048, N=8192, R=64, n=4, reqs=7, none=0, mixed=False),
        # a short training micro-batch on one expert-sized projection
        dict(name="lora_backward 509x2048x512 r16", op="lora_backward", T=509, K=2048, N=512, R=16, n=2, reqs=3, none=0, mixed=False),
        # a training step of several adapters at once
        dict(name="lora_backward 8192x2048x2048 r32", op="lora_backward", T=8192, K=2048, N=2048, R=32, n=6, reqs=16, none=1, mixed=False),
        # a small layer's balance loss over one short batch: latency
        dict(name="balance 300x16 k2", op="balance", T=300, E=16, k=2, n_seq=1, pad=0),
        # a training batch of many tokens in ragged sequences, with padding
        dict(name="balance 65536x256 k6", op="balance", T=65536, E=256, k=6, n_seq=37, pad=9),
        # gradient of the loss alone, odd sizes
        dict(name="balance_backward 2111x200 k5", op="balance_backward", T=2111, E=200, k=5, n_seq=3, pad=4, dw=False),
        # the whole router gradient of a training batch
        dict(name="balance_backward 65536x256 k6", op="balance_backward", T=65536, E=256, k=6, n_seq=37, pad=9, dw=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemv_lora", "lora", "lora", "lora_backward", "balance", "balance_backward"])
    if op == "gemv_lora":
        T = rng.randint(1, 32)
        N, K = rng.choice([(2048, 2048), (2048, 8192), (8192, 2048), (4096, 512), (1040, 768), (272, 4096)])
        return dict(op=op, T=T, K=K, N=N, R=8 * _log_int(rng, 1, 16), n=_log_int(rng, 1, 64), none=rng.randint(0, T // 4),
                    fmt=rng.choice(["nvfp4", "nvfp4", "bf16"]))
    if op in ("lora", "lora_backward"):
        K, N = (8 * _log_int(rng, 16, 1024) for _ in range(2))
        R = 8 * _log_int(rng, 1, 16)
        # no more than the largest listed case of its kind moves and computes
        top = 8192 * (2048 + 2 * 8192) if op == "lora" else 8192 * (3 * 2048 + 2048)
        most = min(8192, top // (K + 2 * N if op == "lora" else 3 * K + N), 8192 * (64 if op == "lora" else 32) * 4096 // (R * (K + N)))
        T = _log_int(rng, 1, max(1, most))
        reqs = min(T, _log_int(rng, 1, 64))
        return dict(op=op, T=T, K=K, N=N, R=R, n=_log_int(rng, 1, 32 if op == "lora" else 8), reqs=reqs,
                    none=rng.randint(0, reqs // 4), mixed=rng.random() < 0.3)
    T = _log_int(rng, 1, 65536)
    E = rng.choice([16, 64, 256, rng.randint(2, 256)])
    case = dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), n_seq=min(T, _log_int(rng, 1, 64)), pad=rng.randint(0, T // 8))
    if op == "balance_backward":
        case["dw"] = rng.random() < 0.7
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _cuts(gen, total, parts):
    """`parts` ragged lengths of at least one that add up to `total` (host integers)."""
    w = torch.rand(parts, generator=gen, dtype=torch.float64) + 0.05
    c = (torch.cumsum(w, 0) / w.sum() * (total - parts)).round().to(torch.int64)
    c = torch.cat([torch.zeros(1, dtype=torch.int64), c])
    return (c[1:] - c[:-1] + 1).tolist()


def _assign(case, gen):
    """Adapter of each token (host int32): whole requests share one, -1 is the base model."""
    T, n = case["T"], case["n"]
    if case["op"] == "gemv_lora":
        lens = [1] * T
    else:
        lens = _cuts(gen, T, case["reqs"])
    order = torch.randperm(n, generator=gen).tolist()
    which = [order[i % n] for i in range(len(lens) - case["none"])] + [-1] * case["none"]
    which = [which[i] for i in torch.randperm(len(which), generator=gen).tolist()]
    adapter = torch.repeat_interleave(torch.tensor(which, dtype=torch.int32), torch.tensor(lens))
    if case.get("mixed"):
        adapter = adapter[torch.randperm(T, generator=gen)]
    return adapter


def _used(case):
    rows = case["T"] if case["op"] == "gemv_lora" else case["reqs"]
    return min(case["n"], rows - case["none"])


def _normal(gen, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * sigma).to(torch.bfloat16)


def _adapters(case, gen):
    K, N, R, n = case["K"], case["N"], case["R"], case["n"]
    return dict(A=_normal(gen, n, R, K, sigma=K ** -0.5), B=_normal(gen, n, N, R, sigma=0.7 * R ** -0.5),
                scale=0.5 + 1.5 * torch.rand(n, generator=gen, device=DEV))


def _projection(case, gen):
    """The shared matrix in its stored form: NVFP4 codes, block scales and tensor scale, or bf16 values."""
    N, K = case["N"], case["K"]
    if case["fmt"] == "bf16":
        return dict(bf16=_normal(gen, N, K, sigma=K ** -0.5))
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device=DEV, dtype=torch.uint8)
    scales = torch.randint(0x30, 0x41, (N, K // 16), generator=gen, device=DEV, dtype=torch.uint8)  # 0.5 .. 2
    return {"codes": codes, "scales": scales, "global": torch.full((1,), 0.3 * K ** -0.5, device=DEV)}


def _dense(src, dtype):
    """The matrix that the stored form stands for, [N][K]."""
    if "bf16" in src:
        return src["bf16"].to(dtype)
    c = src["codes"]
    table = torch.tensor(E2M1, dtype=dtype, device=DEV)
    v = table[torch.stack([c & 15, c >> 4], dim=2).reshape(c.shape[0], -1).long()]
    s = src["scales"].view(torch.float8_e4m3fn).to(torch.float32).to(dtype)
    return v * s.repeat_interleave(16, dim=1) * src["global"].to(dtype)


def _router(case, gen, host):
    """Logits with popular and unpopular experts, the k picks of each token, sequence starts, padding."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=gen, device=DEV) + 0.5 * torch.randn(E, generator=gen, device=DEV)
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    at = torch.tensor([0] + _cuts(host, T, case["n_seq"])).cumsum(0)
    if case["pad"]:
        idx[torch.randperm(T, generator=host)[: case["pad"]].to(DEV)] = -1
    s = dict(logits=logits, idx=idx.contiguous(), seq=at.to(torch.int32).to(DEV), n_seq=case["n_seq"], E=E, k=k, T=T, alpha=1e-2)
    if case["op"] == "balance_backward":
        s["dloss"] = torch.full((1,), 1.0, device=DEV)
        s["dw"] = torch.randn(T, k, generator=gen, device=DEV) / T if case["dw"] else None
        s["seq_counts"], s["seq_tokens"] = _counts(s)  # what the forward call left
    return s


def _inputs(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op = case["op"]
    if op.startswith("balance"):
        return dict(_router(case, gen, host), op=op)
    s = dict(_adapters(case, gen), op=op, T=case["T"], K=case["K"], N=case["N"], R=case["R"], n=case["n"])
    adapter = _assign(case, host)
    s["most"] = max(1, int(torch.bincount((adapter + 1).long(), minlength=2)[1:].max()))  # a scheduler knows its batch
    s["adapter"] = adapter.to(DEV)
    s["x"] = _normal(gen, case["T"], case["K"])
    if op == "gemv_lora":
        s["src"] = _projection(case, gen)
    elif op == "lora":
        s["y"] = _normal(gen, case["T"], case["N"])
    else:
        s["dy"] = _normal(gen, case["T"], case["N"])
        s["dx"] = _normal(gen, case["T"], case["K"])  # the shared projection's part of the gradient
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if s["op"] == "gemv_lora" and not own:
        s["W"] = _dense(s["src"], torch.float32)
    if own:
        _handles(s, case)
    return s


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _handles(s, case):
    """The handles, packed weights, workspaces and output buffers that a program keeps."""
    from w4a16_moe_decode_gb300 import binding as fb
    s["fb"] = fb
    empty = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    if s["op"].startswith("balance"):
        s["cfg"] = fb.make_config(hidden=2048, num_experts=s["E"], top_k=s["k"])
        if s["op"] == "balance":
            s["ws"] = empty(fb.flint_moe_balance_workspace_bytes(s["cfg"], s["T"], s["n_seq"]), dtype=torch.uint8)
            s["out"] = dict(loss=empty(1, dtype=torch.float32), counts=empty(s["E"], dtype=torch.int32),
                            seq_counts=empty(s["n_seq"], s["E"], dtype=torch.int32), seq_tokens=empty(s["n_seq"], dtype=torch.int32))
        else:
            s["out"] = torch.zeros(s["T"], s["E"], device=DEV)
        return
    T, K, N = s["T"], s["K"], s["N"]
    s["lora"] = fb.flint_lora_init(s["A"], s["B"], s["scale"])
    if s["op"] == "gemv_lora":
        s["fmt"] = fb.NVFP4 if case["fmt"] == "nvfp4" else fb.BF16
        s["packed"] = empty(fb.flint_gemv_packed_bytes(N, K, s["fmt"]), dtype=torch.uint8)
        fb.flint_gemv_pack(s["src"], N, K, s["fmt"], s["packed"])
        s["ws"] = empty(fb.flint_gemv_lora_workspace_bytes(s["lora"], T), dtype=torch.uint8)
        s["out"] = empty(T, N)
    elif s["op"] == "lora":
        s["ws"] = empty(fb.flint_lora_workspace_bytes(s["lora"], T), dtype=torch.uint8)
        s["out"] = empty(T, N)
    else:
        s["ws"] = empty(fb.flint_lora_backward_workspace_bytes(s["lora"], T), dtype=torch.uint8)
        s["out"] = dict(dx=empty(T, K), dA=torch.empty_like(s["A"]), dB=torch.empty_like(s["B"]))


def _own(s):
    fb, op, out = s["fb"], s["op"], s["out"]
    if op == "gemv_lora":
        fb.flint_gemv_lora(s["packed"], s["N"], s["K"], s["fmt"], s["x"], s["T"], out, s["lora"], s["adapter"], s["ws"])
    elif op == "lora":
        fb.flint_lora_apply(s["lora"], s["x"], s["adapter"], s["T"], s["y"], out, s["ws"])
    elif op == "lora_backward":
        fb.flint_lora_backward(s["lora"], s["x"], s["dy"], s["adapter"], s["T"], s["dx"], out["dx"], out["dA"], out["dB"], s["ws"])
    elif op == "balance":
        fb.flint_moe_balance(s["cfg"], s["logits"], s["idx"], s["T"], s["seq"], s["n_seq"], s["alpha"], out["loss"], out["counts"],
                             out["seq_counts"], out["seq_tokens"], s["ws"])
    else:
        fb.flint_moe_balance_backward(s["cfg"], s["logits"], s["idx"], s["T"], s["seq"], s["n_seq"], s["alpha"], s["seq_counts"],
                                      s["seq_tokens"], s["dloss"], s["dw"], out)
    return out


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _groups(s):
    """Tokens in order of their adapter, and each one's place in a grid [n][most] (one trash row behind it)."""
    n, most = s["n"], s["most"]
    a = torch.where(s["adapter"] < 0, n, s["adapter"].long())
    order = torch.argsort(a, stable=True)
    a = a[order]
    count = (a[None, :] == torch.arange(n + 1, device=DEV)[:, None]).sum(1)
    first = torch.cumsum(count, 0) - count
    place = torch.arange(s["T"], device=DEV) - first[a]
    return order, torch.where(a < n, a * most + place, n * most)


def _spread(s, v, order, flat):
    g = torch.zeros(s["n"] * s["most"] + 1, v.shape[1], device=DEV)
    g[flat] = v[order].float()
    return g[:-1].view(s["n"], s["most"], -1)


def _add_back(base, d, order, flat):
    """base (fp32 [T][D]) plus the grid's rows; the trash row adds nothing."""
    d = torch.cat([d.reshape(-1, d.shape[2]), torch.zeros(1, d.shape[2], device=DEV)])
    out = base.clone()
    out[order] += d[flat]
    return out.to(torch.bfloat16)


def _plain_lora(s, base):
    order, flat = _groups(s)
    h = torch.bmm(_spread(s, s["x"], order, flat), s["A"].float().transpose(1, 2))
    d = torch.bmm(h, s["B"].float().transpose(1, 2)) * s["scale"][:, None, None]
    return _add_back(base, d, order, flat)


def _plain_lora_backward(s):
    order, flat = _groups(s)
    x, dy = _spread(s, s["x"], order, flat), _spread(s, s["dy"], order, flat)
    A, B = s["A"].float(), s["B"].float()
    h = torch.bmm(x, A.transpose(1, 2)) * s["scale"][:, None, None]
    g = torch.bmm(dy, B) * s["scale"][:, None, None]
    dx = _add_back(s["dx"].float(), torch.bmm(g, A), order, flat)
    return dict(dx=dx, dA=torch.bmm(g.transpose(1, 2), x).to(torch.bfloat16), dB=torch.bmm(dy.transpose(1, 2), h).to(torch.bfloat16))


def _sequence(s):
    """Sequence of each token, and whether it counts."""
    t = torch.arange(s["T"], device=DEV, dtype=torch.int32)
    return torch.bucketize(t, s["seq"][1:], right=True), s["idx"][:, 0] >= 0


def _counts(s):
    seq, counts_in = _sequence(s)
    flat = torch.where(counts_in[:, None], seq[:, None] * s["E"] + s["idx"], s["n_seq"] * s["E"]).long().reshape(-1)
    one = torch.ones_like(flat, dtype=torch.int32)
    c = torch.zeros(s["n_seq"] * s["E"] + 1, dtype=torch.int32, device=DEV).index_add_(0, flat, one)[:-1].view(s["n_seq"], s["E"])
    return c, c.sum(1, dtype=torch.int32) // s["k"]


def _load(s, seq_counts, seq_tokens):
    """f - 1 of each sequence and expert: the share of picks against an even share (whole numbers subtracted, so nothing is lost)."""
    even = (seq_tokens * s["k"]).clamp(min=1)
    return (seq_counts * s["E"] - (seq_tokens * s["k"])[:, None]).float() / even.float()[:, None]


def _plain_balance(s):
    seq_counts, seq_tokens = _counts(s)
    seq, valid = _sequence(s)
    f = _load(s, seq_counts, seq_tokens)
    sg = 1.0 / (1.0 + torch.exp(-s["logits"]))
    p = sg / sg.sum(1, keepdim=True)
    per = torch.where(valid, 1.0 + (f[seq] * p).sum(1), 0.0).double() / seq_tokens[seq].clamp(min=1)
    loss = (per.sum() * (s["alpha"] / s["n_seq"])).float().reshape(1)
    return dict(loss=loss, counts=seq_counts.sum(0, dtype=torch.int32), seq_counts=seq_counts, seq_tokens=seq_tokens)


def _plain_balance_backward(s):
    seq, valid = _sequence(s)
    f = _load(s, s["seq_counts"], s["seq_tokens"])[seq]
    sg = 1.0 / (1.0 + torch.exp(-s["logits"]))
    p = sg / sg.sum(1, keepdim=True)
    c = s["dloss"] * (s["alpha"] / s["n_seq"]) / s["seq_tokens"][seq].clamp(min=1)
    d = c[:, None] * p * (f - (f * p).sum(1, keepdim=True))
    if s["dw"] is not None:
        at = s["idx"].clamp(min=0).long()
        w = torch.gather(sg, 1, at)
        w = w / w.sum(1, keepdim=True)
        d = d.scatter_add(1, at, w * (s["dw"] - (s["dw"] * w).sum(1, keepdim=True)))
    return torch.where(valid[:, None], d * (1.0 / (1.0 + torch.exp(s["logits"]))), 0.0)


def run(s):
    if own:
        return _own(s)
    op = s["op"]
    if op == "gemv_lora":
        return _plain_lora(s, s["x"].float() @ s["W"].T)
    if op == "lora":
        return _plain_lora(s, s["y"].float())
    if op == "lora_backward":
        return _plain_lora_backward(s)
    return _plain_balance(s) if op == "balance" else _plain_balance_backward(s)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op, T = case["op"], case["T"]
    if op.startswith("balance"):
        E, k, n = case["E"], case["k"], case["n_seq"]
        nbytes = 4 * (T * E + T * k + n + 1)
        if op == "balance":
            return {"bytes": nbytes + 4 * (1 + E + n * E + n), "flops": 8 * T * E}
        return {"bytes": nbytes + 4 * (T * E + n * E + n) + (4 * T * k if case["dw"] else 0), "flops": 12 * T * E}
    K, N, R, used = case["K"], case["N"], case["R"], _used(case)
    weights = 2 * used * R * (K + N) + 4 * T + 4 * case["n"]
    if op == "gemv_lora":
        w = N * K * 2 if case["fmt"] == "bf16" else N * K // 2 + N * K // 16 + 4
        return {"bytes": w + weights + 2 * T * (K + N), "flops": 2 * T * N * K + 2 * T * R * (K + N)}
    if op == "lora":
        return {"bytes": weights + 2 * T * (K + 2 * N), "flops": 2 * T * R * (K + N)}
    return {"bytes": weights + 2 * case["n"] * R * (K + N) + 2 * T * (3 * K + N), "flops": 2 * T * R * (3 * K + 2 * N)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_lora(s, base):
    x, A, B = s["x"].double(), s["A"].double(), s["B"].double()
    y = base.clone()
    for a in range(s["n"]):
        rows = torch.nonzero(s["adapter"] == a)[:, 0]
        y[rows] += s["scale"][a].double() * (x[rows] @ A[a].T @ B[a].T)
    return y


def _exact_lora_backward(s):
    x, dy, A, B = s["x"].double(), s["dy"].double(), s["A"].double(), s["B"].double()
    dx, dA, dB = s["dx"].double(), torch.zeros_like(A), torch.zeros_like(B)
    for a in range(s["n"]):
        rows = torch.nonzero(s["adapter"] == a)[:, 0]
        d = s["scale"][a].double() * dy[rows]
        dx[rows] += d @ B[a] @ A[a]
        dA[a] = (d @ B[a]).T @ x[rows]
        dB[a] = d.T @ (x[rows] @ A[a].T)
    return dict(dx=dx, dA=dA, dB=dB)


def _exact_balance(s):
    """Loss, counts and the loss's gradient, one sequence at a time; p is the softmax of log sigmoid(z)."""
    z, at, E, k = s["logits"].double(), s["seq"].tolist(), s["E"], s["k"]
    loss, dz = torch.zeros((), dtype=torch.float64, device=DEV), torch.zeros_like(z)
    seq_counts = torch.zeros(s["n_seq"], E, dtype=torch.int32, device=DEV)
    seq_tokens = torch.zeros(s["n_seq"], dtype=torch.int32, device=DEV)
    for b in range(s["n_seq"]):
        rows = at[b] + torch.nonzero(s["idx"][at[b]:at[b + 1], 0] >= 0)[:, 0]
        seq_tokens[b] = len(rows)
        if not len(rows):
            continue
        seq_counts[b] = torch.bincount(s["idx"][rows].reshape(-1), minlength=E).to(torch.int32)
        f = seq_counts[b].double() * E / (k * len(rows))
        p = torch.softmax(torch.nn.functional.logsigmoid(z[rows]), dim=1)
        c = s["alpha"] / s["n_seq"]
        loss += c * (f * p.mean(0)).sum()
        dz[rows] = c / len(rows) * p * (f - (p * f).sum(1, keepdim=True)) * torch.sigmoid(-z[rows])
    return loss, dz, seq_counts, seq_tokens


def exact(case, seed):
    s = _inputs(case, seed)
    op = s["op"]
    if op == "gemv_lora":
        return _exact_lora(s, s["x"].double() @ _dense(s["src"], torch.float64).T)
    if op == "lora":
        return _exact_lora(s, s["y"].double())
    if op == "lora_backward":
        return _exact_lora_backward(s)
    loss, dz, seq_counts, seq_tokens = _exact_balance(s)
    if op == "balance":
        return dict(loss=loss.reshape(1), counts=seq_counts.sum(0, dtype=torch.int32), seq_counts=seq_counts, seq_tokens=seq_tokens)
    dz = dz * s["dloss"].double()
    if s["dw"] is not None:
        rows = torch.nonzero(s["idx"][:, 0] >= 0)[:, 0]
        at = s["idx"][rows].long()
        sg = torch.sigmoid(s["logits"][rows].double())
        sel = torch.gather(sg, 1, at)
        total = sel.sum(1, keepdim=True)
        dw = s["dw"][rows].double()
        ds = dw / total - (dw * sel).sum(1, keepdim=True) / total ** 2
        part = torch.zeros_like(sg).scatter_add(1, at, ds) * sg * (1 - sg)
        dz[rows] += part
    return dz

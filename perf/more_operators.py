"""Measured cases of the dense gated feed-forward block (decode, many tokens, gradients) and of the orthogonalised
update of matrices that are trained.

Each case is one call a program makes:
  gemv_glu         h = silu(W_g x) * (W_u x) for up to 32 rows on a packed NVFP4 or BF16 pair of matrices
  ffn              y = W_d (silu(W_g x) * (W_u x)) for many tokens on BF16 weights, with (save) the products that the
                   gradients need
  ffn_backward     dx, dW_g, dW_u and dW_d of the same from dy and the saved products
  orthogonalize    Newton-Schulz steps X <- a X + (b X X^T + c (X X^T)^2) X on a batch of matrices, from X / (|X| + eps)

`run` computes them from elementary torch operations in 32 bits, or, where `own` is true, by the library.
"""
import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
STEPS = ((3.4445, -4.7750, 2.0315),) * 5  # the polynomial of each step: singular values in (0, 1] end between 0.7 and 1.2
EPS = 1e-7
NORM_EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoding request in a dense layer of the stack: latency
        dict(name="gemv_glu 1x2048x8192 nvfp4", op="gemv_glu", T=1, K=2048, I=8192, fmt="nvfp4", norm=True),
        # a decode batch on an expert-sized block in the BF16 checkpoint, odd row count
        dict(name="gemv_glu 7x2048x512 bf16", op="gemv_glu", T=7, K=2048, I=512, fmt="bf16", norm=False),
        # the largest decode batch in a dense layer
        dict(name="gemv_glu 32x2048x8192 nvfp4", op="gemv_glu", T=32, K=2048, I=8192, fmt="nvfp4", norm=True),
        # a few requests' tokens past the decode path, in a dense layer: the weights count
        dict(name="ffn 77x2048x8192", op="ffn", T=77, H=2048, I=8192, save=False),
        # a short prompt, odd sizes
        dict(name="ffn 509x1000x2040", op="ffn", T=509, H=1000, I=2040, save=False),
        # the forward pass of a training step, which keeps what the gradients need
        dict(name="ffn 8192x2048x8192 save", op="ffn", T=8192, H=2048, I=8192, save=True),
        # gradients of a short micro-batch on an expert-sized block
        dict(name="ffn_backward 777x2048x512", op="ffn_backward", T=777, H=2048, I=512),
        # gradients of a training step in a dense layer
        dict(name="ffn_backward 8192x2048x8192", op="ffn_backward", T=8192, H=2048, I=8192),
        # the updates of eight adapters of rank 16
        dict(name="orthogonalize 8x16x2048 bf16", op="orthogonalize", n=8, rows=16, cols=2048, dtype="bf16"),
        # the update of a router
        dict(name="orthogonalize 1x256x2048", op="orthogonalize", n=1, rows=256, cols=2048, dtype="f32"),
        # a pair of tall matrices of odd sizes
        dict(name="orthogonalize 2x1001x333", op="orthogonalize", n=2, rows=1001, cols=333, dtype="f32"),
        # the updates of a dense layer's gate and up matrices
        dict(name="orthogonalize 2x8192x2048", op="orthogonalize", n=2, rows=8192, cols=2048, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gemv_glu", "ffn", "ffn", "ffn_backward", "ffn_backward", "orthogonalize", "orthogonalize"])
    if op == "gemv_glu":
        K = rng.choice([256, 512, 768, 1024, 1280, 2048, 2048, 4096, 8192])
        return dict(op=op, T=rng.randint(1, 32), K=K, I=8 * _log_int(rng, 8, min(1024, 2 ** 21 // K)),
                    fmt=rng.choice(["nvfp4", "bf16"]), norm=rng.random() < 0.5)
    if op in ("ffn", "ffn_backward"):
        H, I = 8 * _log_int(rng, 16, 512), 8 * _log_int(rng, 16, 1024)
        # no more than the largest listed case of its kind computes
        case = dict(op=op, T=_log_int(rng, 1, min(8192, 8192 * 2048 * 8192 // (H * I))), H=H, I=I)
        if op == "ffn":
            case["save"] = rng.random() < 0.5
        return case
    rows, cols = _log_int(rng, 8, 4096), _log_int(rng, 8, 8192)
    m, k = min(rows, cols), max(rows, cols)
    top = 2 * (3 * 2048 ** 2 * 8192 + 2048 ** 3)
    return dict(op=op, n=_log_int(rng, 1, max(1, min(64, top // (3 * m * m * k + m ** 3), 2 ** 26 // (m * k)))), rows=rows,
                cols=cols, dtype=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normal(gen, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * sigma).to(torch.bfloat16)


def _projection(fmt, N, K, gen):
    """A matrix in its stored form: NVFP4 codes, block scales and tensor scale, or bf16 values."""
    if fmt == "bf16":
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


def _inputs(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    op = case["op"]
    if op == "orthogonalize":
        # a gradient's momentum: a few strong directions, fading, over noise
        n, rows, cols = case["n"], case["rows"], case["cols"]
        r = min(32, rows, cols)
        fade = torch.exp(-torch.arange(r, device=DEV) / 4.0)
        m = torch.randn(n, rows, r, generator=gen, device=DEV) * fade @ torch.randn(n, r, cols, generator=gen, device=DEV)
        m = 1e-3 * (m + 0.2 * torch.randn(n, rows, cols, generator=gen, device=DEV))
        return dict(op=op, m=m.to(torch.bfloat16) if case["dtype"] == "bf16" else m)
    T = case["T"]
    if op == "gemv_glu":
        K, I = case["K"], case["I"]
        s = dict(op=op, T=T, K=K, I=I, x=_normal(gen, T, K), gate=_projection(case["fmt"], I, K, gen),
                 up=_projection(case["fmt"], I, K, gen))
        s["norm"] = (1.0 + 0.1 * torch.randn(K, generator=gen, device=DEV)).to(torch.bfloat16) if case["norm"] else None
        return s
    H, I = case["H"], case["I"]
    s = dict(op=op, T=T, H=H, I=I, save=case.get("save", False), x=_normal(gen, T, H), gate=_normal(gen, I, H, sigma=H ** -0.5),
             up=_normal(gen, I, H, sigma=H ** -0.5), down=_normal(gen, H, I, sigma=I ** -0.5))
    if op == "ffn_backward":
        s["dy"] = _normal(gen, T, H, sigma=1e-3)
        s["g"] = (s["x"].float() @ s["gate"].float().T).to(torch.bfloat16)  # what the forward pass kept
        s["u"] = (s["x"].float() @ s["up"].float().T).to(torch.bfloat16)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if s["op"] == "gemv_glu" and not own:
        s["Wg"], s["Wu"] = _dense(s["gate"], torch.float32), _dense(s["up"], torch.float32)
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
    op = s["op"]
    if op == "gemv_glu":
        s["fmt"] = fb.NVFP4 if case["fmt"] == "nvfp4" else fb.BF16
        s["packed"] = empty(fb.flint_gemv_glu_packed_bytes(s["I"], s["K"], s["fmt"]), dtype=torch.uint8)
        fb.flint_gemv_glu_pack(s["gate"], s["up"], s["I"], s["K"], s["fmt"], s["packed"])
        s["out"] = empty(s["T"], s["I"])
        return
    if op == "orthogonalize":
        n, rows, cols = s["m"].shape
        s["out"] = empty(n, rows, cols)
        s["ws"] = empty(fb.flint_orthogonalize_workspace_bytes(n, rows, cols), dtype=torch.uint8)
        return
    T, H, I = s["T"], s["H"], s["I"]
    s["ffn"] = fb.flint_ffn_init(s["gate"], s["up"], s["down"])
    if op == "ffn":
        s["ws"] = empty(fb.flint_ffn_workspace_bytes(s["ffn"], T), dtype=torch.uint8)
        s["out"] = dict(y=empty(T, H))
        if s["save"]:
            s["out"].update(g=empty(T, I), u=empty(T, I))
    else:
        s["ws"] = empty(fb.flint_ffn_backward_workspace_bytes(s["ffn"], T), dtype=torch.uint8)
        s["out"] = dict(dx=empty(T, H), dgate=empty(I, H), dup=empty(I, H), ddown=empty(H, I))


def _own(s):
    fb, op, out = s["fb"], s["op"], s["out"]
    if op == "gemv_glu":
        fb.flint_gemv_glu(s["packed"], s["I"], s["K"], s["fmt"], s["x"], s["T"], out, s["norm"], NORM_EPS)
    elif op == "ffn":
        fb.flint_ffn_forward(s["ffn"], s["x"], s["T"], out["y"], s["ws"], out.get("g"), out.get("u"))
    elif op == "ffn_backward":
        fb.flint_ffn_backward(s["ffn"], s["x"], s["g"], s["u"], s["dy"], s["T"], out["dx"], out["dgate"], out["dup"],
                              out["ddown"], s["ws"])
    else:
        fb.flint_orthogonalize(s["m"], out, STEPS, EPS, s["ws"])
    return out


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _bf(t):
    return t.to(torch.bfloat16)


def _plain_glu(s):
    x = s["x"].float()
    if s["norm"] is not None:
        x = _bf(x / torch.sqrt((x * x).mean(1, keepdim=True) + NORM_EPS) * s["norm"].float()).float()  # a rounding of the block
    g, u = x @ s["Wg"].T, x @ s["Wu"].T
    return _bf(g / (1.0 + torch.exp(-g)) * u)


def _plain_ffn(s):
    x = s["x"].float()
    g, u = x @ s["gate"].float().T, x @ s["up"].float().T
    y = (g / (1.0 + torch.exp(-g)) * u) @ s["down"].float().T
    return dict(y=_bf(y), g=_bf(g), u=_bf(u)) if s["save"] else dict(y=_bf(y))


def _plain_ffn_backward(s):
    x, g, u, dy = s["x"].float(), s["g"].float(), s["u"].float(), s["dy"].float()
    dh = dy @ s["down"].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    h = g * sg
    du = dh * h
    dg = dh * u * (sg * (1.0 + g * (1.0 - sg)))
    h = h * u
    dx = dg @ s["gate"].float() + du @ s["up"].float()
    return dict(dx=_bf(dx), dgate=_bf(dg.T @ x), dup=_bf(du.T @ x), ddown=_bf(dy.T @ h))


def _plain_orthogonalize(s):
    x = s["m"].float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (torch.sqrt((x * x).sum(dim=(1, 2), keepdim=True)) + EPS)
    for a, b, c in STEPS:
        g = x @ x.transpose(1, 2)
        x = a * x + (b * g + c * (g @ g)) @ x
    return _bf(x.transpose(1, 2).contiguous() if tall else x)


def run(s):
    if own:
        return _own(s)
    plain = dict(gemv_glu=_plain_glu, ffn=_plain_ffn, ffn_backward=_plain_ffn_backward, orthogonalize=_plain_orthogonalize)
    return plain[s["op"]](s)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "orthogonalize":
        n, m, k = case["n"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # X X^T and its square are symmetric: half of each; the product with X is whole
        return {"bytes": n * m * k * ((4 if case["dtype"] == "f32" else 2) + 2), "flops": n * len(STEPS) * (3 * m * m * k + m ** 3)}
    T, I = case["T"], case["I"]
    if op == "gemv_glu":
        K = case["K"]
        w = 4 * I * K if case["fmt"] == "bf16" else 2 * (I * K // 2 + I * K // 16 + 4)
        return {"bytes": w + 2 * T * (K + I) + (2 * K if case["norm"] else 0), "flops": 4 * T * I * K}
    H = case["H"]
    if op == "ffn":
        return {"bytes": 6 * H * I + 4 * T * H + (4 * T * I if case["save"] else 0), "flops": 6 * T * H * I}
    return {"bytes": 12 * H * I + 6 * T * H + 4 * T * I, "flops": 12 * T * H * I}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_glu(s):
    x = s["x"].double()
    if s["norm"] is not None:
        rms = x.pow(2).sum(1).div(s["K"]).add(NORM_EPS).sqrt()
        x = (x * s["norm"].double() / rms[:, None]).to(torch.bfloat16).double()
    both = x @ torch.cat([_dense(s["gate"], torch.float64), _dense(s["up"], torch.float64)]).T
    g, u = both[:, : s["I"]], both[:, s["I"]:]
    return g * torch.sigmoid(g) * u


def _exact_ffn(s):
    both = s["x"].double() @ torch.cat([s["gate"], s["up"]]).double().T
    g, u = both[:, : s["I"]].contiguous(), both[:, s["I"]:].contiguous()
    y = (g * torch.sigmoid(g) * u) @ s["down"].double().T
    return dict(y=y, g=g, u=u) if s["save"] else dict(y=y)


def _exact_ffn_backward(s):
    """The gradient of sum(dy * y) by automatic differentiation, the products g and u given."""
    w = {k: s[k].double() for k in ("x", "gate", "up", "down", "dy")}
    g, u = s["g"].double().requires_grad_(), s["u"].double().requires_grad_()
    h = g * torch.sigmoid(g) * u
    h.backward(w["dy"] @ w["down"])
    return dict(dx=g.grad @ w["gate"] + u.grad @ w["up"], dgate=g.grad.T @ w["x"], dup=u.grad.T @ w["x"],
                ddown=w["dy"].T @ h.detach())


def _exact_orthogonalize(s):
    out = []
    for m in s["m"]:
        x = m.double()
        x = x / (torch.linalg.matrix_norm(x) + EPS)
        eye = torch.eye(min(x.shape), dtype=torch.float64, device=DEV)
        for a, b, c in STEPS:
            if x.shape[0] <= x.shape[1]:
                g = x @ x.T
                x = (a * eye + (b * eye + c * g) @ g) @ x
            else:
                g = x.T @ x
                x = x @ (a * eye + g @ (b * eye + c * g))
        out.append(x)
    return torch.stack(out)


def exact(case, seed):
    s = _inputs(case, seed)
    return dict(gemv_glu=_exact_glu, ffn=_exact_ffn, ffn_backward=_exact_ffn_backward, orthogonalize=_exact_orthogonalize)[s["op"]](s)

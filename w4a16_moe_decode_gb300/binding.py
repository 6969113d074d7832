"""ctypes binding of libflint_moe.so: the C entry points under the same names.

Argument marshalling only: tensors become device pointers, streams become
cudaStream_t handles, and a non-OK status becomes a FlintMoeError. Every step
of the computation runs in the library's CUDA kernels. If the library has not
been built the first call raises; nothing falls back to another
implementation.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

from .build import LIB

c_int32 = ctypes.c_int32
c_int64 = ctypes.c_int64
c_void_p = ctypes.c_void_p
c_size_t = ctypes.c_size_t

STATUS_NAMES = {0: "FLINT_MOE_OK", 1: "FLINT_MOE_EINVAL", 2: "FLINT_MOE_EALIGN", 3: "FLINT_MOE_ECUDA",
                4: "FLINT_MOE_ETIMEOUT", 5: "FLINT_MOE_EUNSUPPORTED"}
OK, EINVAL, EALIGN, ECUDA, ETIMEOUT, EUNSUPPORTED = range(6)
NVFP4, BF16 = 0, 1
DEV_ERR_TIMEOUT, DEV_ERR_NAN_SCALE, DEV_ERR_SLOTS = 1, 2, 4

# synth tensor tags (same numbering as the CPU generator)
ROUTER, GATE, UP, DOWN, X, BIAS, NORM = 1, 2, 3, 4, 5, 6, 7


class FlintMoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS_NAMES.get(status, status)}")
        self.status = status


class flint_moe_config(ctypes.Structure):
    _fields_ = [("hidden", c_int32), ("num_experts", c_int32), ("top_k", c_int32), ("inter", c_int32),
                ("n_shared", c_int32), ("weight_fmt", c_int32), ("renormalize", c_int32),
                ("routed_scale", ctypes.c_float)]


class flint_moe_nvfp4_src(ctypes.Structure):
    _fields_ = [("codes", c_void_p), ("scales", c_void_p), ("global_", c_void_p)]


class flint_moe_src(ctypes.Structure):
    _fields_ = [("gate", flint_moe_nvfp4_src), ("up", flint_moe_nvfp4_src), ("down", flint_moe_nvfp4_src),
                ("gate_bf16", c_void_p), ("up_bf16", c_void_p), ("down_bf16", c_void_p)]


class flint_lora(ctypes.Structure):
    _fields_ = [("in_dim", c_int32), ("out_dim", c_int32), ("rank", c_int32), ("num_adapters", c_int32),
                ("a", c_void_p), ("b", c_void_p), ("scale", c_void_p)]


class flint_ffn(ctypes.Structure):
    _fields_ = [("hidden", c_int32), ("inter", c_int32), ("gate", c_void_p), ("up", c_void_p), ("down", c_void_p)]


class flint_gemv_src(ctypes.Structure):
    _fields_ = [("codes", c_void_p), ("scales", c_void_p), ("global_", c_void_p), ("bf16", c_void_p)]


class flint_moe_layer(ctypes.Structure):
    _fields_ = [("cfg", flint_moe_config), ("packed", c_void_p), ("router", c_void_p), ("sel_bias", c_void_p),
                ("norm_weight", c_void_p), ("norm_eps", ctypes.c_float)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it was never built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"{LIB} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(LIB)
        P = ctypes.POINTER
        sig = {
            "flint_moe_check_config": (c_int32, [P(flint_moe_config)]),
            "flint_moe_packed_bytes": (c_size_t, [P(flint_moe_config)]),
            "flint_moe_workspace_bytes": (c_size_t, [P(flint_moe_config), c_int32]),
            "flint_moe_workspace_init": (c_int32, [P(flint_moe_config), c_int32, c_void_p, c_void_p]),
            "flint_moe_pack": (c_int32, [P(flint_moe_config), P(flint_moe_src), c_void_p, c_size_t, c_void_p, c_void_p]),
            "flint_moe_unpack_debug": (c_int32, [P(flint_moe_config), c_void_p, P(flint_moe_src), c_void_p]),
            "flint_moe_layer_init": (c_int32, [P(flint_moe_config), c_void_p, c_void_p, c_void_p, P(flint_moe_layer)]),
            "flint_moe_decode": (c_int32, [P(flint_moe_layer), c_void_p, c_int32, c_void_p, c_void_p, c_void_p]),
            "flint_moe_layer_set_norm": (c_int32, [P(flint_moe_layer), c_void_p, ctypes.c_float]),
            "flint_moe_decode_prenorm": (c_int32, [P(flint_moe_layer), c_void_p, c_int32, c_void_p, c_void_p,
                                                   c_void_p]),
            "flint_moe_decode_noalloc": (c_int32, [P(flint_moe_layer), c_void_p, c_int32, c_void_p, c_void_p,
                                                   c_void_p]),
            "flint_moe_debug_routing": (c_int32, [P(flint_moe_config), c_void_p, c_int32, c_void_p, c_void_p, c_void_p]),
            "flint_moe_debug_dequant": (c_int32, [P(flint_moe_config), c_void_p, c_int32, c_int32, c_void_p, c_void_p]),
            "flint_moe_read_status": (c_int32, [c_void_p, P(c_int32), c_void_p]),
            "flint_moe_trace": (c_int32, [c_int32, c_void_p, c_void_p]),
            "flint_moe_debug_rcp_check": (c_int32, [ctypes.c_uint32, ctypes.c_uint32, P(ctypes.c_uint64), c_void_p]),
            "flint_moe_debug_wait_timeout": (c_int32, [c_void_p, c_void_p]),
            "flint_moe_quantize_nvfp4": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p,
                                                   c_void_p]),
            "flint_gemv_packed_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
            "flint_gemv_pack": (c_int32, [P(flint_gemv_src), c_int32, c_int32, c_int32, c_void_p, c_size_t, c_void_p,
                                          c_void_p]),
            "flint_gemv_unpack_debug": (c_int32, [c_void_p, c_int32, c_int32, c_int32, P(flint_gemv_src), c_void_p]),
            "flint_gemv": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int32, c_void_p, c_void_p,
                                     ctypes.c_float, c_void_p, c_void_p]),
            "flint_moe_prefill_workspace_bytes": (c_size_t, [P(flint_moe_config), c_int32]),
            "flint_moe_prefill_workspace_init": (c_int32, [P(flint_moe_config), c_int32, c_void_p, c_void_p]),
            "flint_moe_prefill": (c_int32, [P(flint_moe_layer), c_void_p, c_int32, c_void_p, c_void_p, c_size_t,
                                            c_void_p]),
            "flint_moe_prefill_prenorm": (c_int32, [P(flint_moe_layer), c_void_p, c_int32, c_void_p, c_void_p,
                                                    c_size_t, c_void_p]),
            "flint_moe_prefill_debug_routing": (c_int32, [P(flint_moe_config), c_void_p, c_int32, c_void_p, c_void_p,
                                                          c_void_p, c_void_p]),
            "flint_lora_init": (c_int32, [c_int32, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p,
                                          P(flint_lora)]),
            "flint_lora_workspace_bytes": (c_size_t, [P(flint_lora), c_int32]),
            "flint_lora_apply": (c_int32, [P(flint_lora), c_void_p, c_int64, c_void_p, c_int32, c_void_p, c_void_p,
                                           c_int64, c_void_p, c_size_t, c_void_p]),
            "flint_gemv_lora_workspace_bytes": (c_size_t, [P(flint_lora), c_int32]),
            "flint_gemv_lora": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int32, c_void_p,
                                          P(flint_lora), c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
            "flint_lora_backward_workspace_bytes": (c_size_t, [P(flint_lora), c_int32]),
            "flint_lora_backward": (c_int32, [P(flint_lora), c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int32,
                                              c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_size_t,
                                              c_void_p]),
            "flint_moe_balance_workspace_bytes": (c_size_t, [P(flint_moe_config), c_int32, c_int32]),
            "flint_moe_balance": (c_int32, [P(flint_moe_config), c_void_p, c_void_p, c_int32, c_void_p, c_int32,
                                            ctypes.c_float, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                            c_size_t, c_void_p]),
            "flint_moe_balance_backward": (c_int32, [P(flint_moe_config), c_void_p, c_void_p, c_int32, c_void_p,
                                                     c_int32, ctypes.c_float, c_void_p, c_void_p, c_void_p, c_void_p,
                                                     c_void_p, c_void_p]),
            "flint_gemv_glu_packed_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
            "flint_gemv_glu_pack": (c_int32, [P(flint_gemv_src), P(flint_gemv_src), c_int32, c_int32, c_int32, c_void_p,
                                              c_size_t, c_void_p, c_void_p]),
            "flint_gemv_glu": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int32, c_void_p, c_void_p,
                                         ctypes.c_float, c_void_p, c_void_p]),
            "flint_ffn_init": (c_int32, [c_int32, c_int32, c_void_p, c_void_p, c_void_p, P(flint_ffn)]),
            "flint_ffn_workspace_bytes": (c_size_t, [P(flint_ffn), c_int32]),
            "flint_ffn_forward": (c_int32, [P(flint_ffn), c_void_p, c_int64, c_int32, c_void_p, c_int64, c_void_p,
                                            c_void_p, c_void_p, c_size_t, c_void_p]),
            "flint_ffn_backward_workspace_bytes": (c_size_t, [P(flint_ffn), c_int32]),
            "flint_ffn_backward": (c_int32, [P(flint_ffn), c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_int64,
                                             c_int32, c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_void_p,
                                             c_size_t, c_void_p]),
            "flint_orthogonalize_workspace_bytes": (c_size_t, [c_int32, c_int32, c_int32]),
            "flint_orthogonalize": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_int32, P(ctypes.c_float), c_int32,
                                              ctypes.c_float, ctypes.c_float, c_void_p, c_void_p, c_size_t, c_void_p]),
            "flint_synth_stream_key": (ctypes.c_uint64, [ctypes.c_uint64, ctypes.c_uint32, ctypes.c_uint32,
                                                         ctypes.c_uint32]),
            "flint_synth_normal": (ctypes.c_int, [ctypes.c_uint64, ctypes.c_uint64, c_size_t, ctypes.c_float, c_int32,
                                                  c_void_p, c_void_p]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_current_stream = None


def _stream(stream) -> int | None:
    if stream is None:
        global _current_stream
        if _current_stream is None:
            import torch
            raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
            if raw and device:  # the handle itself: building a Stream object around it takes 3 us of a 5 us call
                torch.cuda.init()
                _current_stream = lambda: raw(device())  # noqa: E731
            else:
                _current_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int) -> None:
    if st != OK:
        raise FlintMoeError(fn, st)


def make_config(hidden=2048, num_experts=256, top_k=6, inter=512, n_shared=1, weight_fmt=NVFP4, renormalize=True,
                routed_scale=1.0) -> flint_moe_config:
    return flint_moe_config(hidden, num_experts, top_k, inter, n_shared, weight_fmt, int(bool(renormalize)),
                            float(routed_scale))


def flint_moe_check_config(cfg: flint_moe_config) -> int:
    return lib().flint_moe_check_config(ctypes.byref(cfg))


def flint_moe_packed_bytes(cfg: flint_moe_config) -> int:
    return lib().flint_moe_packed_bytes(ctypes.byref(cfg))


def flint_moe_workspace_bytes(cfg: flint_moe_config, max_batch: int) -> int:
    return lib().flint_moe_workspace_bytes(ctypes.byref(cfg), max_batch)


def flint_moe_workspace_init(cfg, max_batch, workspace, stream=None) -> None:
    _check("flint_moe_workspace_init",
           lib().flint_moe_workspace_init(ctypes.byref(cfg), max_batch, _ptr(workspace), _stream(stream)))


def _src_struct(src: dict) -> flint_moe_src:
    s = flint_moe_src()
    for m in ("gate", "up", "down"):
        part = getattr(s, m)
        part.codes = _ptr(src.get(m + "_codes"))
        part.scales = _ptr(src.get(m + "_scales"))
        part.global_ = _ptr(src.get(m + "_global"))
        setattr(s, m, part)
        setattr(s, m + "_bf16", _ptr(src.get(m + "_bf16")))
    return s


def flint_moe_pack(cfg, src: dict, dst, dev_status=None, stream=None, dst_bytes=None) -> None:
    """src: dict with keys {gate,up,down}_{codes,scales,global} or {gate,up,down}_bf16 (tensors)."""
    s = _src_struct(src)
    nbytes = dst.numel() * dst.element_size() if dst_bytes is None else dst_bytes
    _check("flint_moe_pack", lib().flint_moe_pack(ctypes.byref(cfg), ctypes.byref(s), _ptr(dst), nbytes,
                                                  _ptr(dev_status), _stream(stream)))


def flint_moe_unpack_debug(cfg, packed, dst: dict, stream=None) -> None:
    s = _src_struct(dst)
    _check("flint_moe_unpack_debug", lib().flint_moe_unpack_debug(ctypes.byref(cfg), _ptr(packed), ctypes.byref(s),
                                                                  _stream(stream)))


def flint_moe_layer_init(cfg, packed, router, sel_bias=None) -> flint_moe_layer:
    layer = flint_moe_layer()
    _check("flint_moe_layer_init", lib().flint_moe_layer_init(ctypes.byref(cfg), _ptr(packed), _ptr(router),
                                                              _ptr(sel_bias), ctypes.byref(layer)))
    return layer


def flint_moe_decode(layer: flint_moe_layer, x, B: int, out, workspace, stream=None) -> None:
    _check("flint_moe_decode", lib().flint_moe_decode(ctypes.byref(layer), _ptr(x), B, _ptr(out), _ptr(workspace),
                                                      _stream(stream)))


def flint_moe_layer_set_norm(layer: flint_moe_layer, norm_weight, eps: float) -> None:
    _check("flint_moe_layer_set_norm", lib().flint_moe_layer_set_norm(ctypes.byref(layer), _ptr(norm_weight),
                                                                      float(eps)))


def flint_moe_decode_prenorm(layer: flint_moe_layer, residual_in, B: int, residual_out, workspace,
                             stream=None) -> None:
    _check("flint_moe_decode_prenorm", lib().flint_moe_decode_prenorm(ctypes.byref(layer), _ptr(residual_in), B,
                                                                      _ptr(residual_out), _ptr(workspace),
                                                                      _stream(stream)))


def flint_moe_decode_noalloc(layer: flint_moe_layer, x, B: int, out, dev_status=None, stream=None) -> None:
    """flint_moe_decode with the library's own 8 MiB device scratch array in
    place of a workspace, for callers that cannot allocate device memory.
    dev_status (int32 device tensor, optional) receives the device status bits."""
    _check("flint_moe_decode_noalloc", lib().flint_moe_decode_noalloc(ctypes.byref(layer), _ptr(x), B, _ptr(out),
                                                                      _ptr(dev_status), _stream(stream)))


def flint_moe_prefill_workspace_bytes(cfg: flint_moe_config, max_tokens: int) -> int:
    return lib().flint_moe_prefill_workspace_bytes(ctypes.byref(cfg), max_tokens)


def flint_moe_prefill_workspace_init(cfg, max_tokens, workspace, stream=None) -> None:
    _check("flint_moe_prefill_workspace_init",
           lib().flint_moe_prefill_workspace_init(ctypes.byref(cfg), max_tokens, _ptr(workspace), _stream(stream)))


def flint_moe_prefill(layer: flint_moe_layer, x, B: int, out, workspace, workspace_bytes=None, stream=None) -> None:
    """The expert-grouped tensor-core path for B tokens (include/flint_moe_prefill.h)."""
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check("flint_moe_prefill", lib().flint_moe_prefill(ctypes.byref(layer), _ptr(x), B, _ptr(out), _ptr(workspace),
                                                        nbytes, _stream(stream)))


def flint_moe_prefill_prenorm(layer: flint_moe_layer, residual_in, B: int, residual_out, workspace,
                              workspace_bytes=None, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check("flint_moe_prefill_prenorm",
           lib().flint_moe_prefill_prenorm(ctypes.byref(layer), _ptr(residual_in), B, _ptr(residual_out),
                                           _ptr(workspace), nbytes, _stream(stream)))


def flint_moe_prefill_debug_routing(cfg, workspace, B, idx, w, logits=None, stream=None) -> None:
    _check("flint_moe_prefill_debug_routing",
           lib().flint_moe_prefill_debug_routing(ctypes.byref(cfg), _ptr(workspace), B, _ptr(idx), _ptr(w),
                                                 _ptr(logits), _stream(stream)))


def flint_moe_debug_routing(cfg, workspace, B, idx, w, stream=None) -> None:
    _check("flint_moe_debug_routing", lib().flint_moe_debug_routing(ctypes.byref(cfg), _ptr(workspace), B, _ptr(idx),
                                                                    _ptr(w), _stream(stream)))


def flint_moe_debug_dequant(cfg, packed, expert, mat, out, stream=None) -> None:
    _check("flint_moe_debug_dequant", lib().flint_moe_debug_dequant(ctypes.byref(cfg), _ptr(packed), expert, mat,
                                                                    _ptr(out), _stream(stream)))


def flint_moe_read_status(workspace, stream=None) -> tuple[int, int]:
    """(status code, device status bits); synchronises the stream."""
    v = c_int32(0)
    st = lib().flint_moe_read_status(_ptr(workspace), ctypes.byref(v), _stream(stream))
    if st not in (OK, ETIMEOUT):
        raise FlintMoeError("flint_moe_read_status", st)
    return st, v.value


def flint_moe_trace(op: int, stream=None):
    """op 0 clears the phase trace; op 1 returns it as a numpy uint64 array
    [64 calls][24 events][2] (earliest, latest ns over blocks). Needs the trace
    build of the library (FLINT_MOE_LIB pointing at it)."""
    import numpy as np
    buf = np.zeros((64, 24, 2), dtype=np.uint64) if op == 1 else None
    st = lib().flint_moe_trace(op, None if buf is None else buf.ctypes.data, _stream(stream))
    _check("flint_moe_trace", st)
    return buf


def flint_moe_debug_rcp_check(lo_bits: int, hi_bits: int, stream=None) -> int:
    """Mismatches between the routing reciprocal and IEEE 1.0f / y over the FP32
    bit patterns [lo_bits, hi_bits) (within [1, 2^125)); synchronises."""
    n = ctypes.c_uint64(0)
    _check("flint_moe_debug_rcp_check", lib().flint_moe_debug_rcp_check(lo_bits, hi_bits, ctypes.byref(n),
                                                                        _stream(stream)))
    return n.value


def flint_moe_debug_wait_timeout(dev_status, stream=None) -> None:
    _check("flint_moe_debug_wait_timeout", lib().flint_moe_debug_wait_timeout(_ptr(dev_status), _stream(stream)))


def flint_moe_quantize_nvfp4(w, n_mat, rows, cols, codes, scales, global_, stream=None) -> None:
    _check("flint_moe_quantize_nvfp4", lib().flint_moe_quantize_nvfp4(_ptr(w), n_mat, rows, cols, _ptr(codes),
                                                                      _ptr(scales), _ptr(global_), _stream(stream)))


def _gemv_src(d: dict) -> flint_gemv_src:
    return flint_gemv_src(_ptr(d.get("codes")), _ptr(d.get("scales")), _ptr(d.get("global")), _ptr(d.get("bf16")))


def flint_gemv_packed_bytes(N: int, K: int, fmt: int = NVFP4) -> int:
    return lib().flint_gemv_packed_bytes(N, K, fmt)


def flint_gemv_pack(src: dict, N: int, K: int, fmt, dst, dev_status=None, stream=None) -> None:
    """src: {codes, scales, global} (NVFP4) or {bf16} tensors of W [N][K]."""
    s = _gemv_src(src)
    _check("flint_gemv_pack", lib().flint_gemv_pack(ctypes.byref(s), N, K, fmt, _ptr(dst),
                                                    dst.numel() * dst.element_size(), _ptr(dev_status),
                                                    _stream(stream)))


def flint_gemv_unpack_debug(packed, N: int, K: int, fmt, dst: dict, stream=None) -> None:
    s = _gemv_src(dst)
    _check("flint_gemv_unpack_debug", lib().flint_gemv_unpack_debug(_ptr(packed), N, K, fmt, ctypes.byref(s),
                                                                    _stream(stream)))


def flint_gemv(packed, N: int, K: int, fmt, x, B: int, y, norm_weight=None, eps: float = 0.0, dev_status=None,
               stream=None) -> None:
    _check("flint_gemv", lib().flint_gemv(_ptr(packed), N, K, fmt, _ptr(x), B, _ptr(y), _ptr(norm_weight),
                                          float(eps), _ptr(dev_status), _stream(stream)))


def _nbytes(workspace, workspace_bytes) -> int:
    return workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes


def _row_stride(t, rows: int, cols: int) -> int | None:
    """Elements between the rows of a tensor of other than two dimensions that holds `rows` rows of `cols` values; None
    if one stride does not describe them."""
    if t.numel() < rows * cols:
        return None
    dims = [(n, st) for n, st in zip(t.shape, t.stride()) if n != 1]
    n = 1  # elements of a row found so far, side by side
    while dims and n < cols and dims[-1][1] == n:
        n *= dims.pop()[0]
    if n != cols:  # also a contiguous buffer that no boundary cuts into rows
        return cols if t.is_contiguous() and (t.dim() < 2 or t.numel() == rows * cols) else None
    for (_, outer), (m, st) in zip(dims, dims[1:]):
        if outer != m * st:
            return None
    return dims[-1][1] if dims and rows > 1 else cols


def _ld(t, rows: int, cols: int, ld, like=None) -> int:
    """Elements between the rows of t: `ld` if given, else a tensor's own row stride (cols where there is one row, no
    tensor or a bare pointer). Refused: elements of a row that do not lie side by side, rows that one stride does not
    describe, fewer of either than are read, and a tensor `like`, read by the same stride, that has another."""
    if ld is not None:
        return ld
    if t is None or isinstance(t, int) or rows < 1:
        return cols
    if t.dim() != 2:
        ld = _row_stride(t, rows, cols)
        if ld is None:
            raise FlintMoeError("rows apart", EINVAL)
    else:
        if t.stride(1) != 1 and cols > 1:
            raise FlintMoeError("row elements apart", EINVAL)
        if t.shape[0] < rows or t.shape[1] < cols:
            raise FlintMoeError("fewer rows or columns", EINVAL)
        ld = cols if rows < 2 else t.stride(0)
    if like is not None and not isinstance(like, int) and like is not t and _ld(like, rows, cols, None) != ld:
        raise FlintMoeError("row strides differ", EINVAL)
    return ld


def _pool(t, shape, bf16: bool, exact: bool) -> None:
    """Refuses a tensor that does not hold an adapter pool's values side by side: bf16 (or their bits) or float32, of
    this shape, or (where the shape was given beside it) at least as many."""
    if t is None or isinstance(t, int):
        return
    import torch
    kinds = (torch.bfloat16, torch.int16, torch.uint16) if bf16 else (torch.float32,)
    if t.dtype not in kinds or not t.is_contiguous() or (tuple(t.shape) != shape if exact else t.numel() < math.prod(shape)):
        raise FlintMoeError(f"adapter pool {tuple(t.shape)} for {shape}", EINVAL)


def flint_lora_init(a, b, scale, in_dim=None, out_dim=None, rank=None, num_adapters=None) -> flint_lora:
    """A pool of adapters: a [n][R][K], b [n][N][R] (bf16), scale [n] (float32), contiguous. The shapes come from the
    tensors unless given. The caller keeps the tensors alive."""
    given = num_adapters is not None
    if not given:
        if a.dim() != 3 or b.dim() != 3:
            raise FlintMoeError("adapter pool", EINVAL)
        num_adapters, rank, in_dim = a.shape
        out_dim = b.shape[1]
    _pool(a, (num_adapters, rank, in_dim), True, not given)
    _pool(b, (num_adapters, out_dim, rank), True, not given)
    _pool(scale, (num_adapters,), False, False)
    lora = flint_lora()
    _check("flint_lora_init", lib().flint_lora_init(in_dim, out_dim, rank, num_adapters, _ptr(a), _ptr(b),
                                                    _ptr(scale), ctypes.byref(lora)))
    return lora


def flint_lora_workspace_bytes(lora: flint_lora, max_tokens: int) -> int:
    return lib().flint_lora_workspace_bytes(ctypes.byref(lora), max_tokens)


def flint_lora_apply(lora: flint_lora, x, adapter, T: int, y_in, y_out, workspace, ldx=None, ldy=None,
                     workspace_bytes=None, stream=None) -> None:
    """y_out[t] = bf16(y_in[t] + scale_a B_a (A_a x[t])), a = adapter[t] (include/flint_lora.h). Row strides
    are those of x and y_out (y_in has to have y_out's)."""
    _check("flint_lora_apply",
           lib().flint_lora_apply(ctypes.byref(lora), _ptr(x), _ld(x, T, lora.in_dim, ldx), _ptr(adapter), T,
                                  _ptr(y_in), _ptr(y_out), _ld(y_out, T, lora.out_dim, ldy, y_in), _ptr(workspace),
                                  _nbytes(workspace, workspace_bytes), _stream(stream)))


def flint_gemv_lora_workspace_bytes(lora: flint_lora, max_batch: int) -> int:
    return lib().flint_gemv_lora_workspace_bytes(ctypes.byref(lora), max_batch)


def flint_gemv_lora(packed, N: int, K: int, fmt, x, B: int, y, lora: flint_lora, adapter, workspace,
                    workspace_bytes=None, dev_status=None, stream=None) -> None:
    """flint_gemv with adapters beside the matrix, one rounding (include/flint_lora.h)."""
    _check("flint_gemv_lora",
           lib().flint_gemv_lora(_ptr(packed), N, K, fmt, _ptr(x), B, _ptr(y), ctypes.byref(lora), _ptr(adapter),
                                 _ptr(workspace), _nbytes(workspace, workspace_bytes), _ptr(dev_status),
                                 _stream(stream)))


def flint_lora_backward_workspace_bytes(lora: flint_lora, max_tokens: int) -> int:
    return lib().flint_lora_backward_workspace_bytes(ctypes.byref(lora), max_tokens)


def flint_lora_backward(lora: flint_lora, x, dy, adapter, T: int, dx_in, dx_out, da, db, workspace, ldx=None,
                        lddy=None, lddx=None, workspace_bytes=None, stream=None) -> None:
    """dx_out, da, db of flint_lora_apply from dy (include/flint_lora.h); dx_out None skips it."""
    _check("flint_lora_backward",
           lib().flint_lora_backward(ctypes.byref(lora), _ptr(x), _ld(x, T, lora.in_dim, ldx), _ptr(dy),
                                     _ld(dy, T, lora.out_dim, lddy), _ptr(adapter), T, _ptr(dx_in), _ptr(dx_out),
                                     _ld(dx_out, T, lora.in_dim, lddx, dx_in), _ptr(da), _ptr(db), _ptr(workspace),
                                     _nbytes(workspace, workspace_bytes), _stream(stream)))


def flint_moe_balance_workspace_bytes(cfg: flint_moe_config, max_tokens: int, max_seqs: int) -> int:
    return lib().flint_moe_balance_workspace_bytes(ctypes.byref(cfg), max_tokens, max_seqs)


def flint_moe_balance(cfg: flint_moe_config, logits, idx, T: int, seq_start, n_seq: int, alpha: float, loss, counts,
                      seq_counts, seq_tokens, workspace, workspace_bytes=None, stream=None) -> None:
    """Balance loss and per-expert counts of T routed tokens (include/flint_moe_balance.h)."""
    _check("flint_moe_balance",
           lib().flint_moe_balance(ctypes.byref(cfg), _ptr(logits), _ptr(idx), T, _ptr(seq_start), n_seq, alpha,
                                   _ptr(loss), _ptr(counts), _ptr(seq_counts), _ptr(seq_tokens), _ptr(workspace),
                                   _nbytes(workspace, workspace_bytes), _stream(stream)))


def flint_moe_balance_backward(cfg: flint_moe_config, logits, idx, T: int, seq_start, n_seq: int, alpha: float,
                               seq_counts, seq_tokens, dloss, dw, dlogits, stream=None) -> None:
    """The logits' gradient of the balance loss and (dw) of the routing weights (include/flint_moe_balance.h)."""
    _check("flint_moe_balance_backward",
           lib().flint_moe_balance_backward(ctypes.byref(cfg), _ptr(logits), _ptr(idx), T, _ptr(seq_start), n_seq,
                                            alpha, _ptr(seq_counts), _ptr(seq_tokens), _ptr(dloss), _ptr(dw),
                                            _ptr(dlogits), _stream(stream)))


@functools.lru_cache(maxsize=None)
def _bf16() -> tuple:
    """The types of tensors that hold bf16 values, or their bits."""
    import torch
    return torch.bfloat16, torch.int16, torch.uint16


def _rows(t, what: str, rows: int, cols: int) -> int | None:
    """The pointer of a tensor that begins with `rows` rows of `cols` bf16 values (or their bits) side by side; others are
    refused."""
    if t is None or isinstance(t, int):
        return t
    shape = t.shape
    n = shape.numel()
    fits = rows < 1 or n == rows * cols or (n > rows * cols and (len(shape) < 2 or shape[-1] == cols))
    if not fits or t.dtype not in _bf16() or not t.is_contiguous():
        raise FlintMoeError(f"{what} {t.dtype} {tuple(shape)} for {(rows, cols)}", EINVAL)
    return t.data_ptr()


def _status_word(t) -> int | None:
    if t is None or isinstance(t, int):
        return t
    import torch
    if t.dtype != torch.int32 or t.numel() < 1:
        raise FlintMoeError(f"status {t.dtype} {tuple(t.shape)}", EINVAL)
    return t.data_ptr()


def _matrix(t, what: str, shape, size: int) -> None:
    """Refuses a tensor of other than `shape` (or its values one behind the other), not contiguous, or whose elements are
    not of `size` bytes (2: bf16 values or their bits)."""
    if t is None or isinstance(t, int):
        return
    flat = t.dim() == 1 and t.numel() == math.prod(shape)
    if t.element_size() != size or (size == 2 and t.dtype not in _bf16()) or not t.is_contiguous() or not (flat or tuple(t.shape) == shape):
        raise FlintMoeError(f"{what} {t.dtype} {tuple(t.shape)} for {shape}", EINVAL)


@functools.lru_cache(maxsize=None)
def _glu_packed_bytes(I: int, K: int, fmt: int) -> int:
    return lib().flint_gemv_glu_packed_bytes(I, K, fmt)


def flint_gemv_glu_packed_bytes(I: int, K: int, fmt: int = NVFP4) -> int:
    return lib().flint_gemv_glu_packed_bytes(I, K, fmt)


def flint_gemv_glu_pack(gate: dict, up: dict, I: int, K: int, fmt, dst, dev_status=None, stream=None) -> None:
    """gate, up: {codes, scales, global} (NVFP4) or {bf16} tensors of matrices [I][K], contiguous."""
    for what, src in (("gate", gate), ("up", up)):
        if fmt == NVFP4:
            _matrix(src.get("codes"), what + " codes", (I, K // 2), 1)
            _matrix(src.get("scales"), what + " scales", (I, K // 16), 1)
            glob = src.get("global")
            if glob is not None and not isinstance(glob, int):
                import torch
                if glob.dtype != torch.float32 or glob.numel() != 1:
                    raise FlintMoeError(f"{what} global {glob.dtype} {tuple(glob.shape)}", EINVAL)
        else:
            _matrix(src.get("bf16"), what, (I, K), 2)
    status = _status_word(dev_status)
    if not dst.is_contiguous():
        raise FlintMoeError("dst", EINVAL)
    g, u = _gemv_src(gate), _gemv_src(up)
    _check("flint_gemv_glu_pack",
           lib().flint_gemv_glu_pack(ctypes.byref(g), ctypes.byref(u), I, K, fmt, _ptr(dst),
                                     dst.numel() * dst.element_size(), status, _stream(stream)))


def flint_gemv_glu(packed, I: int, K: int, fmt, x, B: int, h, norm_weight=None, eps: float = 0.0, dev_status=None,
                   stream=None) -> None:
    """h = bf16(silu(gate x) * (up x)) for up to 32 rows (include/flint_gemv.h): x and h begin with B contiguous rows of K
    and I values."""
    need = _glu_packed_bytes(I, K, fmt) if B > 0 else 0
    # Decode calls are a few microseconds apart and every look at a tensor takes a tenth of one: what they bring as a rule
    # first, with as few looks as tell.
    try:
        plain = (x.dtype is h.dtype is _bf16()[0] and x.nbytes == 2 * B * K and h.nbytes == 2 * B * I and packed.nbytes >= need
                 and x.is_contiguous() and h.is_contiguous() and packed.is_contiguous())
    except AttributeError:  # pointers
        plain = False
    if plain:
        px, ph, pp = x.data_ptr(), h.data_ptr(), packed.data_ptr()
    else:
        px, ph, pp = _rows(x, "x", B, K), _rows(h, "h", B, I), packed
        if not (pp is None or isinstance(pp, int)):
            if pp.nbytes < need or not pp.is_contiguous():
                raise FlintMoeError(f"packed matrices {tuple(pp.shape)}", EINVAL)
            pp = pp.data_ptr()
    if norm_weight is not None:
        norm_weight = _rows(norm_weight, "norm weight", 1, K)
    if dev_status is not None:
        dev_status = _status_word(dev_status)
    st = lib().flint_gemv_glu(pp, I, K, fmt, px, B, ph, norm_weight, float(eps), dev_status, _stream(stream))
    if st != OK:
        raise FlintMoeError("flint_gemv_glu", st)


def _values(t, what: str, shape, bf16: bool = True) -> None:
    """Refuses a tensor that does not hold these values side by side: bf16 (or their bits) or float32, of this shape."""
    if t is None or isinstance(t, int):
        return
    import torch
    kinds = _bf16() if bf16 else (torch.float32,)
    if t.dtype not in kinds or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise FlintMoeError(f"{what} {t.dtype} {tuple(t.shape)} for {tuple(shape)}", EINVAL)


def flint_ffn_init(gate, up, down, hidden=None, inter=None) -> flint_ffn:
    """A dense gated block: gate, up [I][H], down [H][I] (bf16, contiguous). The shapes come from the tensors unless
    given. The caller keeps the tensors alive."""
    if hidden is None or inter is None:
        if gate.dim() != 2:
            raise FlintMoeError("gate", EINVAL)
        inter, hidden = gate.shape
    _values(gate, "gate", (inter, hidden))
    _values(up, "up", (inter, hidden))
    _values(down, "down", (hidden, inter))
    ffn = flint_ffn()
    _check("flint_ffn_init", lib().flint_ffn_init(hidden, inter, _ptr(gate), _ptr(up), _ptr(down), ctypes.byref(ffn)))
    return ffn


def _tokens(**rows) -> None:
    """Refuses tensors of token rows that hold other than bf16 values or their bits (their strides: _ld)."""
    for what, t in rows.items():
        if not (t is None or isinstance(t, int)) and t.dtype not in _bf16():
            raise FlintMoeError(f"{what} {t.dtype}", EINVAL)


def flint_ffn_workspace_bytes(ffn: flint_ffn, max_tokens: int) -> int:
    return lib().flint_ffn_workspace_bytes(ctypes.byref(ffn), max_tokens)


def flint_ffn_forward(ffn: flint_ffn, x, T: int, y, workspace, gate_out=None, up_out=None, ldx=None, ldy=None,
                      workspace_bytes=None, stream=None) -> None:
    """y[t] = down(silu(gate x[t]) * (up x[t])) for T tokens (include/flint_ffn.h). gate_out, up_out [T][I] receive
    what the gradients need."""
    _tokens(x=x, y=y)
    _values(gate_out, "gate_out", (T, ffn.inter))
    _values(up_out, "up_out", (T, ffn.inter))
    _check("flint_ffn_forward",
           lib().flint_ffn_forward(ctypes.byref(ffn), _ptr(x), _ld(x, T, ffn.hidden, ldx), T, _ptr(y),
                                   _ld(y, T, ffn.hidden, ldy), _ptr(gate_out), _ptr(up_out), _ptr(workspace),
                                   _nbytes(workspace, workspace_bytes), _stream(stream)))


def flint_ffn_backward_workspace_bytes(ffn: flint_ffn, max_tokens: int) -> int:
    return lib().flint_ffn_backward_workspace_bytes(ctypes.byref(ffn), max_tokens)


def flint_ffn_backward(ffn: flint_ffn, x, gate_act, up_act, dy, T: int, dx, dgate, dup, ddown, workspace, ldx=None,
                       lddy=None, lddx=None, workspace_bytes=None, stream=None) -> None:
    """Gradients of flint_ffn_forward from dy and the products it kept (include/flint_ffn.h). dx None skips it; dgate,
    dup and ddown None skip the weights'."""
    _tokens(x=x, dy=dy, dx=dx)
    _values(gate_act, "gate_act", (T, ffn.inter))
    _values(up_act, "up_act", (T, ffn.inter))
    _values(dgate, "dgate", (ffn.inter, ffn.hidden))
    _values(dup, "dup", (ffn.inter, ffn.hidden))
    _values(ddown, "ddown", (ffn.hidden, ffn.inter))
    _check("flint_ffn_backward",
           lib().flint_ffn_backward(ctypes.byref(ffn), _ptr(x), _ld(x, T, ffn.hidden, ldx), _ptr(gate_act), _ptr(up_act),
                                    _ptr(dy), _ld(dy, T, ffn.hidden, lddy), T, _ptr(dx), _ld(dx, T, ffn.hidden, lddx),
                                    _ptr(dgate), _ptr(dup), _ptr(ddown), _ptr(workspace),
                                    _nbytes(workspace, workspace_bytes), _stream(stream)))


def flint_orthogonalize_workspace_bytes(n_mat: int, rows: int, cols: int) -> int:
    return lib().flint_orthogonalize_workspace_bytes(n_mat, rows, cols)


def flint_orthogonalize(m, out, coeffs, eps: float, workspace, scale: float = 1.0, workspace_bytes=None,
                        stream=None) -> None:
    """out = bf16(scale X) after the Newton-Schulz steps `coeffs` ((a, b, c) each) from X = m / (|m| + eps), for a matrix
    or a batch of them, float32 or bf16, contiguous (include/flint_orthogonalize.h)."""
    import torch
    f32 = m.dtype == torch.float32
    shape = tuple(m.shape)
    if m.dim() not in (2, 3):
        raise FlintMoeError("matrices", EINVAL)
    _values(m, "matrices", shape, not f32)
    _values(out, "out", shape)
    n, rows, cols = shape if len(shape) == 3 else (1, *shape)
    flat = [float(v) for step in coeffs for v in step]
    if any(len(step) != 3 for step in coeffs):
        raise FlintMoeError("coefficients", EINVAL)
    _check("flint_orthogonalize",
           lib().flint_orthogonalize(_ptr(m), 0 if f32 else 1, n, rows, cols, (ctypes.c_float * len(flat))(*flat),
                                     len(coeffs), float(eps), float(scale), _ptr(out), _ptr(workspace),
                                     _nbytes(workspace, workspace_bytes), _stream(stream)))


def flint_synth_stream_key(seed, layer, tensor, expert) -> int:
    return lib().flint_synth_stream_key(seed, layer, tensor, expert)


def flint_synth_normal(key, start, n, sigma, out_bf16, out, stream=None) -> None:
    st = lib().flint_synth_normal(key, start, n, sigma, int(bool(out_bf16)), _ptr(out), _stream(stream))
    if st != 0:
        raise FlintMoeError("flint_synth_normal", st)

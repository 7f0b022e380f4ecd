"""GB300 (sm_103a) routing-and-combine path of a decode-step latent-MoE layer.

A thin ctypes binding over ``libmoe_decode.so`` (C ABI in ``include/moe_decode.h``):
it checks torch tensors (device, dtype, shape, contiguity), passes their device
pointers and the current CUDA stream, and turns status codes into exceptions. Every
step of the path runs in the library's CUDA kernels; there is no fallback.

BF16 tensors are ``torch.bfloat16``; E4M3 / E8M0 outputs are ``torch.uint8``.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

__all__ = [
    "MoeError", "load", "router_logits", "router_logits_workspace", "front_projection",
    "front_projection_workspace", "topk_route",
    "build_routing_lists", "build_routing_lists_workspace", "unit_windows", "unit_windows_capacity",
    "mxfp8_quantize_rows", "mxfp8_quantize_rows_tcgen05", "mxfp8_tcgen05_scales_bytes",
    "finalize", "finalize_rmsnorm", "route_finalize", "route_finalize_workspace", "device_error", "RouteFinalize",
    "ROUTER_AUTO", "ROUTER_SIMT", "ROUTER_TCGEN05", "MXFP8_SCALE_FLOOR", "MXFP8_SCALE_CEIL",
    "DEVERR_ROW_INDEX", "DEVERR_EXPERT_ID", "DEVERR_TIMEOUT", "DEVERR_CAPACITY",
    "topk_route_grouped", "fp8_block_quantize_rows", "fp8_block_quantize_swiglu", "fp8_block_gemm", "expert_gemm",
    "expert_gemm_workspace",
    "block_norm", "FP8_BLOCK", "SCORE_SIGMOID", "SCORE_SOFTMAX", "GROUP_MAX", "GROUP_TOP2", "FP8_SCALE_AMAX",
    "FP8_SCALE_POW2", "ROWS_TOKEN", "ROWS_LIST", "ROWS_PAIR",
]

OK, ERR_INVALID_ARGUMENT, ERR_ALIGNMENT, ERR_CAPACITY, ERR_WORKSPACE, ERR_UNSUPPORTED, ERR_CUDA = range(7)
DEVERR_ROW_INDEX, DEVERR_EXPERT_ID, DEVERR_TIMEOUT, DEVERR_CAPACITY = 0x1, 0x2, 0x4, 0x8
ROUTER_AUTO, ROUTER_SIMT, ROUTER_TCGEN05 = 0, 1, 2
MXFP8_SCALE_FLOOR, MXFP8_SCALE_CEIL = 0, 1
DTYPE_F32, DTYPE_BF16 = 0, 1
FP8_BLOCK = 128
SCORE_SIGMOID, SCORE_SOFTMAX = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1
FP8_SCALE_AMAX, FP8_SCALE_POW2 = 0, 1
ROWS_TOKEN, ROWS_LIST, ROWS_PAIR = 0, 1, 2
GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_FULL = 0, 1, 2, 3

# Every symbol the header declares, with its ctypes signature.
_P, _I, _SZ, _F, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_int64
SIGNATURES = {
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_version": (_I, []),
    "moe_device_error": (_I, [ctypes.POINTER(ctypes.c_uint32), _I]),
    "moe_router_logits_workspace": (_SZ, [_I, _I, _I]),
    "moe_router_logits": (_I, [_P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "moe_router_logits_ex": (_I, [_P, _P, _P, _I, _I, _I, _P, _SZ, _I, _P]),
    "moe_router_logits_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _P]),
    "moe_front_projection_workspace": (_SZ, [_I, _I, _I, _I]),
    "moe_front_projection": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "moe_topk_route": (_I, [_P, _P, _I, _I, _I, _I, _F, _P, _P, _P, _P]),
    "moe_topk_route_quantize": (_I, [_P, _P, _I, _I, _I, _I, _F, _P, _P, _P, _P, _I, _I, _P, _P, _P]),
    "moe_build_routing_lists_workspace": (_SZ, [_I, _I, _I]),
    "moe_build_routing_lists": (_I, [_P, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "moe_unit_windows_capacity": (_I, [_I, _I, _I, _I]),
    "moe_build_unit_windows": (_I, [_P, _I, _I, _P, _P, _P, _P, _I, _P]),
    "mxfp8_quantize_rows": (_I, [_P, _I, _I, _P, _P, _P]),
    "mxfp8_quantize_rows_ex": (_I, [_P, _I, _I, _P, _P, _I, _P]),
    "mxfp8_tcgen05_scales_bytes": (_SZ, [_I, _I]),
    "mxfp8_quantize_rows_tcgen05": (_I, [_P, _I, _I, _P, _P, _I, _P]),
    "moe_finalize": (_I, [_P, ctypes.c_int64, _P, _P, _I, _P, _F, _I, _I, _I, _P, _P]),
    "moe_finalize_rmsnorm": (_I, [_P, ctypes.c_int64, _P, _P, _I, _F, _P, _F, _I, _I, _I, _P, _P, _P]),
    "moe_route_finalize_workspace": (_SZ, [_I, _I, _I, _I]),
    "moe_route_finalize": (_I, [_P] * 5 + [_I] * 6 + [_F] + [_P] * 9 + [_P, _SZ, _P]),
    "moe_topk_route_grouped": (_I, [_P, _P] + [_I] * 8 + [_F, _P, _P, _P, _P]),
    "fp8_block_quantize_rows": (_I, [_P, _L, _I, _I, _P, _P, _I, _P]),
    "fp8_block_quantize_swiglu": (_I, [_P, _L, _I, _I, _P, _P, _I, _P]),
    "fp8_block_gemm": (_I, [_P] * 5 + [_I] * 4 + [_P]),
    "moe_expert_gemm_workspace": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_expert_gemm": (_I, [_P, _P, _L, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "moe_block_norm": (_I, [_P, _L, _P, _I, _P, _P, _I, _P, _F, _F, _I, _I, _P, _P, _P, _P, _P]),
}

_lib = None


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = load().moe_status_string(status).decode()
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


def load(path: str | None = None):
    """Load the CUDA library (built in-tree by ``build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build the CUDA library first (latent_moe_decode_gb300.build.build())")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != OK:
        raise MoeError(fn, status)


def _stream(stream):
    # (the current stream's handle without its Python object: 0.3 instead of 3 us a call)
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, dtype, shape=None, name="tensor"):
    try:  # (a torch.Size compares as the tuple that it is)
        if t.dtype is dtype and (shape is None or t.shape == shape) and t.is_contiguous() and t.is_cuda:
            return t
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _empty(shape, dtype, like, stream=None):
    """A new tensor for a launch on `stream`: of that stream's memory, so that it is neither still in
    use by the current stream's earlier work nor, once dropped, handed to its later work while the
    launch runs; the current stream may use it as well."""
    if stream is not None:
        current = torch.cuda.current_stream(like.device)
        if stream.cuda_stream != current.cuda_stream:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream.cuda_stream, device=like.device)):
                t = torch.empty(shape, dtype=dtype, device=like.device)
            t.record_stream(current)
            return t
    return torch.empty(shape, dtype=dtype, device=like.device)


def _scratch(workspace, need, like, stream):
    """(workspace, its bytes): the caller's, of any type and shape, or a new one of `need` bytes (None for 0)."""
    if workspace is None:
        return (_empty((need,), torch.uint8, like, stream), need) if need else (None, 0)
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace: expected a torch.Tensor")
    if not workspace.is_cuda and workspace.numel():
        raise ValueError("workspace: must be a CUDA tensor")
    if not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


# ---------------------------------------------------------------------------
def router_logits_workspace(T: int, H: int, E: int) -> int:
    return int(load().moe_router_logits_workspace(T, H, E))


def router_logits(x, w, out=None, workspace=None, algo: int = ROUTER_AUTO, stream=None):
    """FP32 logits [T, E] = x [T, H] (BF16) @ w [E, H]^T (BF16)."""
    T, H = x.shape
    E = w.shape[0]
    _need(x, torch.bfloat16, (T, H), "x")
    _need(w, torch.bfloat16, (E, H), "w")
    out = _empty((T, E), torch.float32, x, stream) if out is None else _need(out, torch.float32, (T, E), "out")
    workspace, wb = _scratch(workspace, router_logits_workspace(T, H, E), x, stream)
    _check("moe_router_logits_ex", load().moe_router_logits_ex(
        _ptr(x), _ptr(w), _ptr(out), T, H, E, _ptr(workspace), wb, algo, _stream(stream)))
    return out


def front_projection_workspace(T: int, H: int, E: int, L: int) -> int:
    return int(load().moe_front_projection_workspace(T, H, E, L))


def front_projection(x, w_router, w_down, logits=None, latent=None, workspace=None, stream=None):
    """(FP32 logits [T, E] = x @ w_router^T, BF16 latent [T, L] = bf16(x @ w_down^T)), one launch."""
    T, H = x.shape
    E, L = w_router.shape[0], w_down.shape[0]
    _need(x, torch.bfloat16, (T, H), "x")
    _need(w_router, torch.bfloat16, (E, H), "w_router")
    _need(w_down, torch.bfloat16, (L, H), "w_down")
    logits = _empty((T, E), torch.float32, x, stream) if logits is None else _need(logits, torch.float32, (T, E), "logits")
    latent = _empty((T, L), torch.bfloat16, x, stream) if latent is None else _need(latent, torch.bfloat16, (T, L), "latent")
    workspace, wb = _scratch(workspace, front_projection_workspace(T, H, E, L), x, stream)
    _check("moe_front_projection", load().moe_front_projection(
        _ptr(x), _ptr(w_router), _ptr(w_down), _ptr(logits), _ptr(latent), T, H, E, L, _ptr(workspace), wb,
        _stream(stream)))
    return logits, latent


def topk_route(logits, bias, K: int, renormalize: bool = True, scale: float = 1.0,
               ids=None, weights=None, weights_bf16=None, want_bf16: bool = True, stream=None):
    """(ids int32 [T,K], weights FP32 [T,K], weights BF16 [T,K] or None)."""
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    ids = _empty((T, K), torch.int32, logits, stream) if ids is None else _need(ids, torch.int32, (T, K), "ids")
    weights = _empty((T, K), torch.float32, logits, stream) if weights is None else _need(weights, torch.float32, (T, K), "weights")
    if weights_bf16 is None and want_bf16:
        weights_bf16 = _empty((T, K), torch.bfloat16, logits, stream)
    elif weights_bf16 is not None:
        _need(weights_bf16, torch.bfloat16, (T, K), "weights_bf16")
    _check("moe_topk_route", load().moe_topk_route(
        _ptr(logits), _ptr(bias), T, E, K, int(bool(renormalize)), float(scale),
        _ptr(ids), _ptr(weights), _ptr(weights_bf16), _stream(stream)))
    return ids, weights, weights_bf16


def topk_route_quantize(logits, bias, K: int, latent, renormalize: bool = True, scale: float = 1.0, ids=None,
                        weights=None, weights_bf16=None, q=None, scales=None, stream=None):
    """topk_route and mxfp8_quantize_rows(latent) in one launch:
    (ids, weights, weights_bf16, q, scales)."""
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    rows, cols = latent.shape
    _need(latent, torch.bfloat16, (rows, cols), "latent")
    ids = _empty((T, K), torch.int32, logits, stream) if ids is None else _need(ids, torch.int32, (T, K), "ids")
    weights = _empty((T, K), torch.float32, logits, stream) if weights is None else _need(weights, torch.float32, (T, K), "weights")
    weights_bf16 = _empty((T, K), torch.bfloat16, logits, stream) if weights_bf16 is None else _need(weights_bf16, torch.bfloat16, (T, K), "weights_bf16")
    q = _empty((rows, cols), torch.uint8, latent, stream) if q is None else _need(q, torch.uint8, (rows, cols), "q")
    scales = _empty((rows, cols // 32), torch.uint8, latent, stream) if scales is None else _need(scales, torch.uint8, (rows, cols // 32), "scales")
    _check("moe_topk_route_quantize", load().moe_topk_route_quantize(
        _ptr(logits), _ptr(bias), T, E, K, int(bool(renormalize)), float(scale), _ptr(ids), _ptr(weights),
        _ptr(weights_bf16), _ptr(latent), rows, cols, _ptr(q), _ptr(scales), _stream(stream)))
    return ids, weights, weights_bf16, q, scales


def build_routing_lists_workspace(T: int, K: int, E: int) -> int:
    return int(load().moe_build_routing_lists_workspace(T, K, E))


def build_routing_lists(ids, E: int, offsets=None, pairs=None, workspace=None, stream=None):
    """CSR lists: offsets int32 [E+1], pairs int32 [T*K] (pair code t*K + k)."""
    T, K = ids.shape
    _need(ids, torch.int32, (T, K), "ids")
    offsets = _empty((E + 1,), torch.int32, ids, stream) if offsets is None else _need(offsets, torch.int32, (E + 1,), "offsets")
    pairs = _empty((T * K,), torch.int32, ids, stream) if pairs is None else _need(pairs, torch.int32, (T * K,), "pairs")
    workspace, wb = _scratch(workspace, build_routing_lists_workspace(T, K, E), ids, stream)
    _check("moe_build_routing_lists", load().moe_build_routing_lists(
        _ptr(ids), T, K, E, _ptr(offsets), _ptr(pairs), _ptr(workspace), wb, _stream(stream)))
    return offsets, pairs


def unit_windows_capacity(T: int, K: int, E: int, window: int = 8) -> int:
    n = int(load().moe_unit_windows_capacity(T, K, E, window))
    if n < 0:
        raise MoeError("moe_unit_windows_capacity", ERR_INVALID_ARGUMENT)
    return n


def unit_windows(offsets, window: int = 8, max_units: int | None = None, unit_offsets=None, unit_expert=None,
                 unit_start=None, unit_len=None, stream=None):
    """Units of `window` listed pairs per expert from CSR offsets int32 [E+1]:
    (unit_offsets [E+1], unit_expert, unit_start, unit_len [max_units]); the first
    unit_offsets[E] entries are the units."""
    E = offsets.shape[0] - 1
    _need(offsets, torch.int32, (E + 1,), "offsets")
    if max_units is None:
        max_units = unit_expert.shape[0] if unit_expert is not None else None
    if max_units is None:
        raise ValueError("max_units (or preallocated unit arrays) required: see unit_windows_capacity()")
    unit_offsets = _empty((E + 1,), torch.int32, offsets, stream) if unit_offsets is None else _need(unit_offsets, torch.int32, (E + 1,), "unit_offsets")
    outs = []
    for t, name in ((unit_expert, "unit_expert"), (unit_start, "unit_start"), (unit_len, "unit_len")):
        if t is None:
            t = _empty((max_units,), torch.int32, offsets, stream)
        elif _need(t, torch.int32, None, name).dim() != 1 or t.shape[0] < max_units:
            raise ValueError(f"{name}: expected a 1-D tensor of at least {max_units} entries")
        outs.append(t)
    _check("moe_build_unit_windows", load().moe_build_unit_windows(
        _ptr(offsets), E, int(window), _ptr(unit_offsets), _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), int(max_units),
        _stream(stream)))
    return (unit_offsets, *outs)


def mxfp8_quantize_rows(x, q=None, scales=None, stream=None, scale_rule: int = MXFP8_SCALE_FLOOR):
    """(E4M3 bytes uint8 [rows, cols], E8M0 scale bytes uint8 [rows, cols/32]);
    scale_rule MXFP8_SCALE_FLOOR (OCP) or MXFP8_SCALE_CEIL (no saturation)."""
    rows, cols = x.shape
    _need(x, torch.bfloat16, (rows, cols), "x")
    q = _empty((rows, cols), torch.uint8, x, stream) if q is None else _need(q, torch.uint8, (rows, cols), "q")
    nb = cols // 32
    scales = _empty((rows, nb), torch.uint8, x, stream) if scales is None else _need(scales, torch.uint8, (rows, nb), "scales")
    _check("mxfp8_quantize_rows_ex", load().mxfp8_quantize_rows_ex(_ptr(x), rows, cols, _ptr(q), _ptr(scales),
                                                                   int(scale_rule), _stream(stream)))
    return q, scales


def mxfp8_tcgen05_scales_bytes(rows: int, cols: int) -> int:
    """Bytes of the tcgen05 block-scaling scale layout of a [rows, cols] MXFP8 tensor."""
    return int(load().mxfp8_tcgen05_scales_bytes(rows, cols))


def mxfp8_quantize_rows_tcgen05(x, q=None, scales=None, stream=None, scale_rule: int = MXFP8_SCALE_FLOOR):
    """(E4M3 bytes uint8 [rows, cols], E8M0 scales uint8 [mxfp8_tcgen05_scales_bytes]
    in the tcgen05 block-scaling tile layout)."""
    rows, cols = x.shape
    _need(x, torch.bfloat16, (rows, cols), "x")
    q = _empty((rows, cols), torch.uint8, x, stream) if q is None else _need(q, torch.uint8, (rows, cols), "q")
    n = mxfp8_tcgen05_scales_bytes(rows, cols)
    scales = _empty((n,), torch.uint8, x, stream) if scales is None else _need(scales, torch.uint8, (n,), "scales")
    _check("mxfp8_quantize_rows_tcgen05", load().mxfp8_quantize_rows_tcgen05(
        _ptr(x), rows, cols, _ptr(q), _ptr(scales), int(scale_rule), _stream(stream)))
    return q, scales


def finalize(rows, weights, T: int, K: int, row_index=None, shared=None, scale: float = 1.0, out=None, stream=None):
    """BF16 out [T, H] = sum_k w[t,k] * rows[r(t,k)] (+ shared[t])."""
    n_rows, H = rows.shape
    _need(rows, torch.bfloat16, (n_rows, H), "rows")
    if weights.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif weights.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError("weights: expected float32 or bfloat16")
    _need(weights, weights.dtype, (T, K), "weights")
    if row_index is not None:
        _need(row_index, torch.int32, (T, K), "row_index")
    if shared is not None:
        _need(shared, torch.bfloat16, (T, H), "shared")
    out = _empty((T, H), torch.bfloat16, rows, stream) if out is None else _need(out, torch.bfloat16, (T, H), "out")
    _check("moe_finalize", load().moe_finalize(
        _ptr(rows), n_rows, _ptr(row_index), _ptr(weights), dt, _ptr(shared), float(scale), T, K, H, _ptr(out),
        _stream(stream)))
    return out


def finalize_rmsnorm(rows, weights, T: int, K: int, norm_weight, eps: float = 1e-5, row_index=None,
                     scale: float = 1.0, routed=None, out=None, want_routed: bool = True, stream=None):
    """(routed BF16 [T, H] or None, RMSNorm(routed) * norm_weight BF16 [T, H])."""
    n_rows, H = rows.shape
    _need(rows, torch.bfloat16, (n_rows, H), "rows")
    if weights.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    elif weights.dtype == torch.float32:
        dt = DTYPE_F32
    else:
        raise TypeError("weights: expected float32 or bfloat16")
    _need(weights, weights.dtype, (T, K), "weights")
    _need(norm_weight, torch.bfloat16, (H,), "norm_weight")
    if row_index is not None:
        _need(row_index, torch.int32, (T, K), "row_index")
    if routed is None and want_routed:
        routed = _empty((T, H), torch.bfloat16, rows, stream)
    elif routed is not None:
        _need(routed, torch.bfloat16, (T, H), "routed")
    out = _empty((T, H), torch.bfloat16, rows, stream) if out is None else _need(out, torch.bfloat16, (T, H), "out")
    _check("moe_finalize_rmsnorm", load().moe_finalize_rmsnorm(
        _ptr(rows), n_rows, _ptr(row_index), _ptr(weights), dt, float(scale), _ptr(norm_weight), float(eps), T, K, H,
        _ptr(routed), _ptr(out), _stream(stream)))
    return routed, out


def device_error(clear: bool = True) -> int:
    """The library's device error word (DEVERR_* bits); synchronises the device."""
    v = ctypes.c_uint32(0)
    _check("moe_device_error", load().moe_device_error(ctypes.byref(v), int(bool(clear))))
    return int(v.value)


def route_finalize_workspace(T: int, H: int, E: int, K: int) -> int:
    return int(load().moe_route_finalize_workspace(T, H, E, K))


def route_finalize(x, w, bias, latent, rows, K: int, renormalize: bool, scale: float, logits, ids, weights,
                   weights_bf16, offsets, pairs, q, scales, out, workspace=None, stream=None):
    """The whole step in one library call (all outputs preallocated): router logits ->
    top-K + MXFP8 -> routing lists -> Finalize of rows [T*K, L] with the BF16 weights."""
    T, H = x.shape
    E = w.shape[0]
    L = latent.shape[1]
    _need(x, torch.bfloat16, (T, H), "x")
    _need(w, torch.bfloat16, (E, H), "w")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    _need(latent, torch.bfloat16, (T, L), "latent")
    _need(rows, torch.bfloat16, (T * K, L), "rows")
    for t, dt, shape, name in ((logits, torch.float32, (T, E), "logits"), (ids, torch.int32, (T, K), "ids"),
                               (weights_bf16, torch.bfloat16, (T, K), "weights_bf16"),
                               (offsets, torch.int32, (E + 1,), "offsets"), (pairs, torch.int32, (T * K,), "pairs"),
                               (q, torch.uint8, (T, L), "q"), (scales, torch.uint8, (T, L // 32), "scales"),
                               (out, torch.bfloat16, (T, L), "out")):
        _need(t, dt, shape, name)
    if weights is not None:
        _need(weights, torch.float32, (T, K), "weights")
    workspace, ws = _scratch(workspace, 0, x, stream)
    _check("moe_route_finalize", load().moe_route_finalize(
        _ptr(x), _ptr(w), _ptr(bias), _ptr(latent), _ptr(rows), T, H, L, E, K, int(bool(renormalize)), float(scale),
        _ptr(logits), _ptr(ids), _ptr(weights), _ptr(weights_bf16), _ptr(offsets), _ptr(pairs), _ptr(q), _ptr(scales),
        _ptr(out), _ptr(workspace), ws, _stream(stream)))
    return out


# --- the experts in 8-bit floating point: E4M3 codes (torch.uint8) with an FP32 scale per
# --- row and 128 columns (activations) or per 128 x 128 block (weights)
def _rows_2d(t, dtype, name):
    """A 2-D CUDA tensor of contiguous rows, `stride(0)` elements apart (a slice of wider rows is one)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected two dimensions and contiguous rows")
    return t


def _row_stride(t):
    """Elements between rows (a single row has any stride: its length then)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def _out_dtype(out, out_dtype):
    dt = out.dtype if out is not None else out_dtype
    if dt == torch.bfloat16:
        return dt, DTYPE_BF16
    if dt == torch.float32:
        return dt, DTYPE_F32
    raise TypeError("out: expected float32 or bfloat16")


def topk_route_grouped(logits, bias, K: int, n_group: int = 1, topk_group: int = 1, scoring: int = SCORE_SIGMOID,
                       group_rule: int = GROUP_TOP2, renormalize: bool = True, scale: float = 1.0, ids=None,
                       weights=None, weights_bf16=None, want_bf16: bool = True, stream=None):
    """(ids int32 [T,K], weights FP32 [T,K], weights BF16 [T,K] or None): sigmoid or softmax
    scores, the choice among the best topk_group of n_group groups of experts."""
    T, E = logits.shape
    _need(logits, torch.float32, (T, E), "logits")
    if bias is not None:
        _need(bias, torch.float32, (E,), "bias")
    ids = _empty((T, K), torch.int32, logits, stream) if ids is None else _need(ids, torch.int32, (T, K), "ids")
    weights = _empty((T, K), torch.float32, logits, stream) if weights is None else _need(weights, torch.float32, (T, K), "weights")
    if weights_bf16 is not None:
        _need(weights_bf16, torch.bfloat16, (T, K), "weights_bf16")
    elif want_bf16:
        weights_bf16 = _empty((T, K), torch.bfloat16, logits, stream)
    _check("moe_topk_route_grouped", load().moe_topk_route_grouped(
        _ptr(logits), _ptr(bias), T, E, K, int(scoring), int(n_group), int(topk_group), int(group_rule),
        int(bool(renormalize)), float(scale), _ptr(ids), _ptr(weights), _ptr(weights_bf16), _stream(stream)))
    return ids, weights, weights_bf16


def _block_quantize(fn, x, cols, q, scales, scale_rule, stream):
    rows = x.shape[0]
    q = _empty((rows, cols), torch.uint8, x, stream) if q is None else _need(q, torch.uint8, (rows, cols), "q")
    nb = _blocks(cols)
    scales = _empty((rows, nb), torch.float32, x, stream) if scales is None else _need(scales, torch.float32, (rows, nb), "scales")
    _check(fn, getattr(load(), fn)(_ptr(x), _row_stride(x), rows, cols, _ptr(q), _ptr(scales), int(scale_rule),
                                   _stream(stream)))
    return q, scales


def fp8_block_quantize_rows(x, q=None, scales=None, scale_rule: int = FP8_SCALE_AMAX, stream=None):
    """(E4M3 codes uint8 [rows, cols], FP32 scales [rows, ceil(cols / 128)]) of BF16 rows
    (contiguous rows; their stride may exceed their length)."""
    _rows_2d(x, torch.bfloat16, "x")
    return _block_quantize("fp8_block_quantize_rows", x, x.shape[1], q, scales, scale_rule, stream)


def fp8_block_quantize_swiglu(gate_up, q=None, scales=None, scale_rule: int = FP8_SCALE_AMAX, stream=None):
    """The codes and scales of silu(gate) * up [rows, F], gate_up BF16 [rows, 2 F] = [gate | up]."""
    _rows_2d(gate_up, torch.bfloat16, "gate_up")
    if gate_up.shape[1] % 2:
        raise ValueError("gate_up: expected an even number of columns")
    return _block_quantize("fp8_block_quantize_swiglu", gate_up, gate_up.shape[1] // 2, q, scales, scale_rule, stream)


def fp8_block_gemm(a, a_scales, w, w_scales, out=None, out_dtype=torch.bfloat16, stream=None):
    """out [M, N] (BF16 or FP32) = codes a [M, K] times codes w [N, K]^T with their scales
    (a_scales FP32 [M, ceil(K/128)], w_scales FP32 [ceil(N/128), ceil(K/128)])."""
    M, K = a.shape
    N = w.shape[0]
    _need(a, torch.uint8, (M, K), "a")
    _need(a_scales, torch.float32, (M, _blocks(K)), "a_scales")
    _need(w, torch.uint8, (N, K), "w")
    _need(w_scales, torch.float32, (_blocks(N), _blocks(K)), "w_scales")
    dt, code = _out_dtype(out, out_dtype)
    out = _empty((M, N), dt, a, stream) if out is None else _need(out, dt, (M, N), "out")
    _check("fp8_block_gemm", load().fp8_block_gemm(_ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales), _ptr(out), code,
                                                   M, N, K, _stream(stream)))
    return out


def expert_gemm_workspace(n_pairs: int, E: int, N: int, K: int, in_rows: int = ROWS_TOKEN) -> int:
    return int(load().moe_expert_gemm_workspace(n_pairs, E, N, K, in_rows))


def expert_gemm(a, a_scales, w, w_scales, offsets, pairs, topk: int, in_rows: int = ROWS_TOKEN,
                out_rows: int = ROWS_PAIR, out=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """out [n_pairs, N] (BF16 or FP32): every listed pair's row of codes a times its expert's
    weights w [E, N, K]^T, over the lists of build_routing_lists (offsets [E+1], pairs).
    in_rows: which row of a a pair multiplies (ROWS_TOKEN, ROWS_LIST, ROWS_PAIR); out_rows:
    which row of out it writes (ROWS_LIST, ROWS_PAIR)."""
    a_rows, K = a.shape
    E, N = w.shape[0], w.shape[1]
    P = pairs.shape[0]
    _need(a, torch.uint8, (a_rows, K), "a")
    _need(a_scales, torch.float32, (a_rows, _blocks(K)), "a_scales")
    _need(w, torch.uint8, (E, N, K), "w")
    _need(w_scales, torch.float32, (E, _blocks(N), _blocks(K)), "w_scales")
    _need(offsets, torch.int32, (E + 1,), "offsets")
    _need(pairs, torch.int32, (P,), "pairs")
    dt, code = _out_dtype(out, out_dtype)
    out = _empty((P, N), dt, a, stream) if out is None else _need(out, dt, (P, N), "out")
    workspace, wb = _scratch(workspace, expert_gemm_workspace(P, E, N, K, in_rows), a, stream)
    _check("moe_expert_gemm", load().moe_expert_gemm(
        _ptr(a), _ptr(a_scales), a_rows, _ptr(w), _ptr(w_scales), _ptr(offsets), _ptr(pairs), P, int(topk), int(in_rows),
        int(out_rows), _ptr(out), code, E, N, K, _ptr(workspace), wb, _stream(stream)))
    return out


def block_norm(y, residual, next_weight, post_weight=None, gate=None, alpha: float = 1.0, eps: float = 1e-6, h=None,
               n=None, quantize: bool = False, q=None, scales=None, stream=None):
    """(h, n, q, scales): h = residual + alpha * gate * rms(y) * post_weight (of the residual's
    dtype, BF16 or FP32), n = rms(h) * next_weight (BF16), and with quantize n's codes and
    scales (else None). gate: BF16 [T, 1], [H] or [T, H]. h may be the residual itself."""
    T, H = residual.shape
    _rows_2d(y, torch.bfloat16, "y")
    if y.shape != (T, H):
        raise ValueError(f"y: expected shape {(T, H)}, got {tuple(y.shape)}")
    dt, code = _out_dtype(residual, None)
    full, row = (T, H), (H,)
    _need(residual, dt, full, "residual")
    _need(next_weight, torch.bfloat16, row, "next_weight")
    if post_weight is not None:
        _need(post_weight, torch.bfloat16, row, "post_weight")
    kind = GATE_NONE
    if gate is not None:
        _need(gate, torch.bfloat16, None, "gate")
        kind = {full: GATE_FULL, row: GATE_CHANNEL, (T, 1): GATE_TOKEN}.get(tuple(gate.shape))
        if kind is None:
            raise ValueError(f"gate: expected shape {(T, 1)}, {row} or {full}, got {tuple(gate.shape)}")
    h = _empty((T, H), dt, y, stream) if h is None else _need(h, dt, (T, H), "h")
    n = _empty((T, H), torch.bfloat16, y, stream) if n is None else _need(n, torch.bfloat16, (T, H), "n")
    if quantize:
        q = _empty((T, H), torch.uint8, y, stream) if q is None else _need(q, torch.uint8, (T, H), "q")
        nb = _blocks(H)
        scales = _empty((T, nb), torch.float32, y, stream) if scales is None else _need(scales, torch.float32, (T, nb), "scales")
    else:
        q = scales = None
    _check("moe_block_norm", load().moe_block_norm(
        _ptr(y), _row_stride(y), _ptr(residual), code, _ptr(post_weight), _ptr(gate), kind, _ptr(next_weight),
        float(alpha), float(eps), T, H, _ptr(h), _ptr(n), _ptr(q), _ptr(scales), _stream(stream)))
    return h, n, q, scales


class RouteFinalize:
    """The whole routing-and-combine step, with its buffers preallocated:
    router logits -> sigmoid+bias top-K with the MXFP8 latent in the same launch ->
    Finalize, whose launch also builds the routing lists (Finalize does not read them),
    on one stream.

    ``run()`` launches the library's kernels (programmatic dependent launch between
    consecutive kernels of a stream) and allocates nothing, so it can be captured in a
    CUDA graph. With the automatic router choice it is one library call
    (``moe_route_finalize``); with a forced router family, the four calls.
    """

    def __init__(self, T: int, H: int, L: int, E: int, K: int, device="cuda", renormalize=True, scale=1.0,
                 router_algo: int = ROUTER_AUTO):
        self.T, self.H, self.L, self.E, self.K = T, H, L, E, K
        self.renormalize, self.scale, self.router_algo = renormalize, scale, router_algo
        dev = torch.device(device)
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=dev)
        self.logits = e((T, E), torch.float32)
        self.ids = e((T, K), torch.int32)
        self.weights = e((T, K), torch.float32)
        self.weights_bf16 = e((T, K), torch.bfloat16)
        self.offsets = e((E + 1,), torch.int32)
        self.pairs = e((T * K,), torch.int32)
        self.q = e((T, L), torch.uint8)
        self.scales = e((T, L // 32), torch.uint8)
        self.out = e((T, L), torch.bfloat16)
        self.router_ws = e((max(1, router_logits_workspace(T, H, E)),), torch.uint8)
        self.lists_ws = e((max(1, build_routing_lists_workspace(T, K, E)),), torch.uint8)
        self.chain_ws = e((max(1, route_finalize_workspace(T, H, E, K)),), torch.uint8)
        self.launches = self._count_launches()

    def _count_launches(self) -> int:
        """Kernels one run() launches."""
        if self.router_algo == ROUTER_AUTO:
            # the one-call step: router (its split-K partials summed by the top-K launch),
            # top-k + MXFP8, Finalize with the routing lists
            return 3
        # the four calls; a forced router family may add its split-K reduce kernel
        return 4 + (1 if router_logits_workspace(self.T, self.H, self.E) > 0 else 0)

    def run(self, x, w, bias, latent, rows, stream=None):
        main = stream if stream is not None else torch.cuda.current_stream()
        if self.router_algo == ROUTER_AUTO:
            return route_finalize(x, w, bias, latent, rows, self.K, self.renormalize, self.scale, self.logits, self.ids,
                                  self.weights, self.weights_bf16, self.offsets, self.pairs, self.q, self.scales,
                                  self.out, workspace=self.chain_ws, stream=main)
        router_logits(x, w, out=self.logits, workspace=self.router_ws, algo=self.router_algo, stream=main)
        topk_route_quantize(self.logits, bias, self.K, latent, self.renormalize, self.scale, ids=self.ids,
                            weights=self.weights, weights_bf16=self.weights_bf16, q=self.q, scales=self.scales,
                            stream=main)
        build_routing_lists(self.ids, self.E, offsets=self.offsets, pairs=self.pairs, workspace=self.lists_ws,
                            stream=main)
        finalize(rows, self.weights_bf16, self.T, self.K, out=self.out, stream=main)
        return self.out

"""Python binding of libnvfp4moe, the NVFP4 block-scaled MoE layer for MI355X.

Argument marshalling only: each function checks tensor devices/dtypes/shapes,
allocates outputs with torch (device memory is all torch is used for), and
calls the C entry point of the same name on the current HIP stream.  Every
step of the computation runs in the library's HIP kernels; there is no CPU or
eager-PyTorch fallback, and importing a function whose library is missing
raises.

C entry points (include/nvfp4moe.h): moe_route_permute, nvfp4_quantize,
nvfp4_grouped_gemm, moe_swiglu, moe_unpermute_combine, moe_route_quantize
(routing and activation quantisation in shared launches) and moe_expert_ffn
(gate_up + SwiGLU requant + down for all experts, one persistent launch at
decode sizes); mxfp4_* and fp8_* variants; moe_gated_ffn and moe_grouped_gemm
with their gradients (16-bit experts); int8_quantize and int8_grouped_gemm;
moe_route_scored (softmax or sigmoid scores, balance bias, expert groups) and
moe_unpermute_combine_backward with their gradients; int4_quantize,
int4_dequantize and int4_grouped_gemv (4-bit weights on 16-bit rows).

With stream=, operands, given results and given workspaces have to be ready on
that stream, and the caller orders it before work that reads the results; the
memory that a call allocates for itself is that stream's and needs no such order.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libnvfp4moe.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = range(5)
F32, BF16, F16 = 0, 1, 2
EPI_F32, EPI_BF16, EPI_SWIGLU_NVFP4, EPI_COMBINE_F32, EPI_SWIGLU_BF16 = range(5)
ACT_SILU, ACT_GELU = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1


class NVFP4MoEError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"nvfp4moe status {status}: {detail}")
        self.status = status
        self.detail = detail


class FfnArgs(ctypes.Structure):
    """Mirror of nvfp4moe_ffn_args."""
    _fields_ = [
        ("x_codes", ctypes.c_void_p), ("x_scales", ctypes.c_void_p), ("x_g", ctypes.c_void_p),
        ("x_rows", ctypes.c_int64), ("perm_src_token", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
        ("E", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("m_total", ctypes.c_int64),
        ("w_gu_packed", ctypes.c_void_p), ("g_gu", ctypes.c_void_p),
        ("w_dn_packed", ctypes.c_void_p), ("g_dn", ctypes.c_void_p), ("g_h", ctypes.c_void_p),
        ("h_codes", ctypes.c_void_p), ("h_scales", ctypes.c_void_p), ("y", ctypes.c_void_p),
        ("max_rows_per_expert_hint", ctypes.c_int32),
        ("out", ctypes.c_void_p), ("perm_of_assignment", ctypes.c_void_p), ("topk_w", ctypes.c_void_p),
        ("T", ctypes.c_int32), ("k", ctypes.c_int32),
    ]


class GemmArgs(ctypes.Structure):
    """Mirror of nvfp4moe_gemm_args."""
    _fields_ = [
        ("a_codes", ctypes.c_void_p), ("a_scales", ctypes.c_void_p), ("a_g", ctypes.c_void_p),
        ("a_rows", ctypes.c_void_p), ("a_rows_total", ctypes.c_int64),
        ("b_codes", ctypes.c_void_p), ("b_scales", ctypes.c_void_p), ("b_g", ctypes.c_void_p),
        ("offsets", ctypes.c_void_p),
        ("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
        ("m_total", ctypes.c_int64), ("epilogue", ctypes.c_int32),
        ("out", ctypes.c_void_p), ("out_rows", ctypes.c_int64),
        ("out_codes", ctypes.c_void_p), ("out_scales", ctypes.c_void_p), ("out_g", ctypes.c_void_p),
        ("row_token", ctypes.c_void_p), ("row_weight", ctypes.c_void_p),
        ("max_rows_per_expert_hint", ctypes.c_int32),
        ("b_packed", ctypes.c_void_p),
    ]


class Fp8GemmArgs(ctypes.Structure):
    """Mirror of nvfp4moe_fp8_gemm_args."""
    _fields_ = [
        ("a_codes", ctypes.c_void_p), ("a_scales", ctypes.c_void_p), ("a_rows", ctypes.c_void_p),
        ("a_rows_total", ctypes.c_int64), ("b_packed", ctypes.c_void_p), ("b_scales", ctypes.c_void_p),
        ("offsets", ctypes.c_void_p), ("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
        ("m_total", ctypes.c_int64), ("epilogue", ctypes.c_int32), ("out", ctypes.c_void_p),
        ("max_rows_per_expert_hint", ctypes.c_int32), ("out_codes", ctypes.c_void_p), ("out_scales", ctypes.c_void_p),
    ]


def _struct(name, doc, fields):
    kinds = {"p": ctypes.c_void_p, "i": ctypes.c_int32, "l": ctypes.c_int64, "f": ctypes.c_float}
    return type(name, (ctypes.Structure,), {"__doc__": doc, "_fields_": [(n, kinds[k]) for n, k in fields]})


GatedArgs = _struct("GatedArgs", "Mirror of nvfp4moe_gated_args.", [
    ("x", "p"), ("dtype", "i"), ("a_rows", "p"), ("x_rows", "l"), ("w", "p"), ("offsets", "p"), ("E", "i"), ("H", "i"),
    ("I", "i"), ("m_total", "l"), ("activation", "i"), ("max_rows_per_expert_hint", "i"), ("h", "p"), ("gu", "p")])
GatedGradArgs = _struct("GatedGradArgs", "Mirror of nvfp4moe_gated_grad_args.", [
    ("x", "p"), ("dtype", "i"), ("a_rows", "p"), ("x_rows", "l"), ("w", "p"), ("offsets", "p"), ("E", "i"), ("H", "i"),
    ("I", "i"), ("m_total", "l"), ("activation", "i"), ("max_rows_per_expert_hint", "i"), ("gu", "p"), ("dh", "p"),
    ("dx", "p"), ("dw", "p")])
ProductArgs = _struct("ProductArgs", "Mirror of nvfp4moe_product_args.", [
    ("a", "p"), ("dtype", "i"), ("a_rows", "p"), ("a_rows_total", "l"), ("b", "p"), ("offsets", "p"), ("E", "i"),
    ("N", "i"), ("K", "i"), ("m_total", "l"), ("out_dtype", "i"), ("max_rows_per_expert_hint", "i"), ("out", "p")])
ProductGradArgs = _struct("ProductGradArgs", "Mirror of nvfp4moe_product_grad_args.", [
    ("a", "p"), ("dtype", "i"), ("a_rows", "p"), ("a_rows_total", "l"), ("b", "p"), ("offsets", "p"), ("E", "i"),
    ("N", "i"), ("K", "i"), ("m_total", "l"), ("max_rows_per_expert_hint", "i"), ("dy", "p"), ("da", "p"), ("db", "p")])
Int8GemmArgs = _struct("Int8GemmArgs", "Mirror of nvfp4moe_int8_gemm_args.", [
    ("a_codes", "p"), ("a_scales", "p"), ("a_rows", "p"), ("a_rows_total", "l"), ("b_codes", "p"), ("b_scales", "p"),
    ("offsets", "p"), ("E", "i"), ("N", "i"), ("K", "i"), ("m_total", "l"), ("epilogue", "i"),
    ("max_rows_per_expert_hint", "i"), ("out", "p")])
RouteArgs = _struct("RouteArgs", "Mirror of nvfp4moe_route_args.", [
    ("logits", "p"), ("dtype", "i"), ("T", "i"), ("E", "i"), ("k", "i"), ("score", "i"), ("renormalize", "i"),
    ("scale", "f"), ("bias", "p"), ("n_group", "i"), ("topk_group", "i"), ("group_top", "i"), ("topk_ids", "p"),
    ("topk_w", "p"), ("counts", "p"), ("offsets", "p"), ("perm_src_token", "p"), ("perm_of_assignment", "p"),
    ("perm_weight", "p"), ("scores", "p")])
RouteGradArgs = _struct("RouteGradArgs", "Mirror of nvfp4moe_route_grad_args.", [
    ("logits", "p"), ("dtype", "i"), ("T", "i"), ("E", "i"), ("k", "i"), ("score", "i"), ("renormalize", "i"),
    ("scale", "f"), ("bias", "p"), ("topk_ids", "p"), ("d_topk_w", "p"), ("d_scores", "p"), ("d_scores_ld", "l"),
    ("dlogits", "p")])
Int4GemvArgs = _struct("Int4GemvArgs", "Mirror of nvfp4moe_int4_gemv_args.", [
    ("a", "p"), ("dtype", "i"), ("a_rows", "p"), ("a_rows_total", "l"), ("b_codes", "p"), ("b_scales", "p"),
    ("b_zeros", "p"), ("group", "i"), ("offsets", "p"), ("E", "i"), ("N", "i"), ("K", "i"), ("m_total", "l"),
    ("gated", "i"), ("activation", "i"), ("out_dtype", "i"), ("max_rows_per_expert_hint", "i"), ("out", "p")])


_lib = None

_SIGNATURES = {
    "moe_route_permute_workspace_size": (ctypes.c_size_t, [ctypes.c_int32] * 3),
    "moe_route_permute": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
                          + [ctypes.c_void_p] * 8 + [ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_quantize_workspace_size": (ctypes.c_size_t, []),
    "nvfp4_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64]
                       + [ctypes.c_void_p] * 5 + [ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(GemmArgs), ctypes.c_void_p]),
    "nvfp4_weight_packed_size": (ctypes.c_size_t, [ctypes.c_int32] * 3),
    "nvfp4_weight_repack": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_swiglu_workspace_size": (ctypes.c_size_t, []),
    "moe_swiglu": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32]
                   + [ctypes.c_void_p] * 5 + [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_unpermute_combine": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                             ctypes.c_int32, ctypes.c_void_p]),
    "moe_route_quantize_workspace_size": (ctypes.c_size_t, [ctypes.c_int32] * 3),
    "moe_route_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
                           + [ctypes.c_void_p] * 7 + [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64]
                           + [ctypes.c_void_p] * 4 + [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_route_quantize_noalloc_max_workspace": (ctypes.c_size_t, []),
    "moe_route_quantize_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
                                   + [ctypes.c_void_p] * 7 + [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64]
                                   + [ctypes.c_void_p] * 4 + [ctypes.c_void_p]),
    "moe_expert_ffn_workspace_size": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                                        ctypes.c_int32]),
    "moe_expert_ffn": (ctypes.c_int, [ctypes.POINTER(FfnArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "mxfp4_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "mxfp4_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(GemmArgs), ctypes.c_void_p]),
    "mxfp4_weight_packed_size": (ctypes.c_size_t, [ctypes.c_int32] * 3),
    "mxfp4_weight_repack": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "fp8_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                    ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "fp8_swiglu_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "fp8_weight_packed_size": (ctypes.c_size_t, [ctypes.c_int32] * 3),
    "fp8_weight_repack": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                         ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "fp8_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(Fp8GemmArgs), ctypes.c_void_p]),
    "moe_gated_ffn": (ctypes.c_int, [ctypes.POINTER(GatedArgs), ctypes.c_void_p]),
    "moe_gated_ffn_backward_workspace_size": (ctypes.c_size_t, [ctypes.c_int32] * 3 + [ctypes.c_int64]),
    "moe_gated_ffn_backward": (ctypes.c_int, [ctypes.POINTER(GatedGradArgs), ctypes.c_void_p, ctypes.c_size_t,
                                              ctypes.c_void_p]),
    "moe_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(ProductArgs), ctypes.c_void_p]),
    "moe_grouped_gemm_backward_workspace_size": (ctypes.c_size_t, [ctypes.c_int32] * 3 + [ctypes.c_int64]),
    "moe_grouped_gemm_backward": (ctypes.c_int, [ctypes.POINTER(ProductGradArgs), ctypes.c_void_p, ctypes.c_size_t,
                                                 ctypes.c_void_p]),
    "int8_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p]),
    "int8_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(Int8GemmArgs), ctypes.c_void_p]),
    "moe_route_scored": (ctypes.c_int, [ctypes.POINTER(RouteArgs), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_route_scored_backward": (ctypes.c_int, [ctypes.POINTER(RouteGradArgs), ctypes.c_void_p]),
    "moe_unpermute_combine_backward": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                                      ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]
                                       + [ctypes.c_int32] * 3 + [ctypes.c_void_p] * 3),
    "int4_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32,
                                     ctypes.c_int32] + [ctypes.c_void_p] * 4),
    "int4_dequantize": (ctypes.c_int, [ctypes.c_void_p] * 3 + [ctypes.c_int64] * 2 + [ctypes.c_int32] * 3
                        + [ctypes.c_void_p] * 2),
    "int4_grouped_gemv": (ctypes.c_int, [ctypes.POINTER(Int4GemvArgs), ctypes.c_void_p]),
    "nvfp4moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "nvfp4moe_last_error_detail": (ctypes.c_char_p, []),
    "nvfp4moe_version": (ctypes.c_int, []),
}


def lib() -> ctypes.CDLL:
    """Load libnvfp4moe.so (built in-tree by block_scaled_fp4_permute_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m block_scaled_fp4_permute_amd.build` "
                              "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != OK:
        detail = lib().nvfp4moe_last_error_detail().decode()
        raise NVFP4MoEError(status, detail)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _call(dev, stream, fn, *args):
    """A C call on ``stream`` (None: the current stream of the operands' device)
    with that device current, whichever one is."""
    import torch
    if stream is not None:
        if getattr(stream, "device", dev) != dev:
            raise ValueError(f"stream: of {stream.device}, the operands are on {dev}")
        raw = stream.cuda_stream
    else:
        raw = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch._C._cuda_getDevice() == dev.index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status:
        _check(status)


def _need(t, dtype, name, device=None):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


_torch = None       # imported with the first allocation: the library itself needs none


def _empty(shape, dtype, dev):
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    if type(shape) is tuple and shape:       # a tuple costs 0.8 us more than its numbers
        return _torch.empty(*shape, dtype=dtype, device=dev)
    return _torch.empty(shape, dtype=dtype, device=dev)


def _new(shape, dtype, dev, stream):
    """Working memory of a call on ``stream`` (None: the current one), from that
    stream's pool.  A block of the current stream's pool may have been freed
    with work still queued there that uses it, and nothing orders that work
    before the call's."""
    if stream is None:
        return _empty(shape, dtype, dev)
    import torch
    with torch.cuda.stream(stream):
        return _empty(shape, dtype, dev)


def _new_result(shape, dtype, dev, stream):
    """Memory for a call's result; the caller reads it on the current stream, for
    which it is held when it is dropped."""
    if stream is None:
        return _empty(shape, dtype, dev)
    import torch
    out = _new(shape, dtype, dev, stream)
    out.record_stream(torch.cuda.current_stream(dev))
    return out


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _dtype_any(t, name):
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return F16
    raise TypeError(f"{name}: expected float32, bfloat16 or float16, got {t.dtype}")


def _need_shape(t, shape, dtype, name, device):
    _need(t, dtype, name, device)
    if t.shape != shape:
        raise ValueError(f"{name}: expected {list(shape)}, got {list(t.shape)}")


# --------------------------------------------------------------------------- route
@dataclass
class Routing:
    topk_ids: "object"
    topk_w: "object"
    counts: "object"
    offsets: "object"
    perm_src_token: "object"
    perm_of_assignment: "object"
    perm_weight: "object"


def _new_routing(T, E, k, dev, stream):
    import torch
    i32, f32 = torch.int32, torch.float32
    if stream is None:
        # of another tensor's type and device: a fifth less than by naming them
        ids, w, n = _empty((T, k), i32, dev), _empty((T, k), f32, dev), T * k
        new = ids.new_empty
        return Routing(ids, w, new(E), new(E + 1), new(n), new(n), w.new_empty(n))
    new = _new_result
    return Routing(new((T, k), i32, dev, stream), new((T, k), f32, dev, stream), new(E, i32, dev, stream),
                   new(E + 1, i32, dev, stream), new(T * k, i32, dev, stream), new(T * k, i32, dev, stream),
                   new(T * k, f32, dev, stream))


def moe_route_permute(logits, k: int, out: Routing | None = None, workspace=None, stream=None) -> Routing:
    """logits float32 [T, E] -> Routing (see include/nvfp4moe.h)."""
    import torch
    _need(logits, torch.float32, "logits")
    T, E = logits.shape
    dev = logits.device
    if out is None:
        out = _new_routing(T, E, k, dev, stream)
    nbytes = lib().moe_route_permute_workspace_size(T, E, k)
    if workspace is None:
        workspace = _new(max(nbytes, 16), torch.uint8, dev, stream)
    _call(dev, stream, lib().moe_route_permute,
          logits.data_ptr(), T, E, k, out.topk_ids.data_ptr(), out.topk_w.data_ptr(), out.counts.data_ptr(),
          out.offsets.data_ptr(), out.perm_src_token.data_ptr(), out.perm_of_assignment.data_ptr(),
          _ptr(out.perm_weight), workspace.data_ptr(), workspace.numel())
    return out


# --------------------------------------------------------------- router with scores
def moe_route_scored(logits, k: int, *, score: int = SCORE_SOFTMAX, bias=None, n_group: int = 1, topk_group: int = 1,
                     group_top: int = 1, renormalize: bool = True, scale: float = 1.0, save_scores: bool = False,
                     scores=None, out: Routing | None = None, workspace=None, stream=None):
    """logits float32/bf16/f16 [T, E] -> Routing by softmax or sigmoid scores, with
    a balance bias float32 [E] on the choice, the topk_group best of n_group expert
    groups, weights renormalised over the k chosen or not, times scale (see
    include/nvfp4moe.h).  save_scores (or a float32 scores [T, E]): returns
    (Routing, scores)."""
    import torch
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    code = _dtype_any(logits, "logits")
    dev = logits.device
    _need(logits, logits.dtype, "logits", dev)
    T, E = logits.shape
    if bias is not None:
        _need_shape(bias, (E,), torch.float32, "bias", dev)
    f32, i32 = torch.float32, torch.int32
    if out is None:
        out = _new_routing(T, E, k, dev, stream)
    else:
        for t, shape, dtype, name in ((out.topk_ids, (T, k), i32, "topk_ids"), (out.topk_w, (T, k), f32, "topk_w"),
                                      (out.counts, (E,), i32, "counts"), (out.offsets, (E + 1,), i32, "offsets"),
                                      (out.perm_src_token, (T * k,), i32, "perm_src_token"),
                                      (out.perm_of_assignment, (T * k,), i32, "perm_of_assignment")):
            _need_shape(t, shape, dtype, "out." + name, dev)
        if out.perm_weight is not None:
            _need_shape(out.perm_weight, (T * k,), f32, "out.perm_weight", dev)
    if save_scores or scores is not None:
        scores = _result(scores, (T, E), f32, logits, "scores", stream)
    ws = _scratch(workspace, lib().moe_route_permute_workspace_size(T, E, k), dev, stream)
    # in the order of the fields
    args = RouteArgs(logits.data_ptr(), code, T, E, k, score, int(renormalize), scale, _ptr(bias), n_group, topk_group,
                     group_top, out.topk_ids.data_ptr(), out.topk_w.data_ptr(), out.counts.data_ptr(),
                     out.offsets.data_ptr(), out.perm_src_token.data_ptr(), out.perm_of_assignment.data_ptr(),
                     _ptr(out.perm_weight), _ptr(scores))
    _call(dev, stream, lib().moe_route_scored, ctypes.byref(args), ws.data_ptr(), ws.numel())
    return out if scores is None else (out, scores)


def moe_route_scored_backward(d_topk_w, logits, topk_ids, *, score: int = SCORE_SOFTMAX, bias=None,
                              renormalize: bool = True, scale: float = 1.0, d_scores=None, dlogits=None, stream=None):
    """Gradient of the logits [T, E], in their type, from d_topk_w float32 [T, k];
    logits, topk_ids and options of the forward call (bias only if it holds -inf or
    NaN).  d_scores: float32 gradient of the scores, [T, E] or one row [E] for all
    tokens."""
    import torch
    if logits.dim() != 2 or topk_ids.dim() != 2:
        raise ValueError("logits must be [T, E] and topk_ids [T, k]")
    code = _dtype_any(logits, "logits")
    dev = logits.device
    _need(logits, logits.dtype, "logits", dev)
    T, E = logits.shape
    k = topk_ids.shape[1]
    _need_shape(topk_ids, (T, k), torch.int32, "topk_ids", dev)
    _need_shape(d_topk_w, (T, k), torch.float32, "d_topk_w", dev)
    if bias is not None:
        _need_shape(bias, (E,), torch.float32, "bias", dev)
    ld = 0
    if d_scores is not None:
        ld = E if d_scores.dim() == 2 else 0
        _need_shape(d_scores, (T, E) if ld else (E,), torch.float32, "d_scores", dev)
    dlogits = _result(dlogits, (T, E), logits.dtype, logits, "dlogits", stream)
    # in the order of the fields
    args = RouteGradArgs(logits.data_ptr(), code, T, E, k, score, int(renormalize), scale, _ptr(bias), topk_ids.data_ptr(),
                         d_topk_w.data_ptr(), _ptr(d_scores), ld, dlogits.data_ptr())
    _call(dev, stream, lib().moe_route_scored_backward, ctypes.byref(args))
    return dlogits


# ------------------------------------------------------------------------ quantise
@dataclass
class NVFP4Tensor:
    codes: "object"     # uint8 [rows, cols/2]
    scales: "object"    # uint8 [rows, cols/16]
    g: "object"         # float32 [1] (device)


def nvfp4_quantize(x, g=None, out: NVFP4Tensor | None = None, workspace=None, stream=None) -> NVFP4Tensor:
    """x bf16/float32 [rows, cols] -> NVFP4Tensor.  g: optional device float32[1]
    per-tensor scale (None: amax/2688 computed on the device)."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    _need(x, x.dtype, "x")
    rows, cols = x.shape
    dev = x.device
    if out is None:
        out = NVFP4Tensor(_new_result((rows, cols // 2), torch.uint8, dev, stream),
                          _new_result((rows, cols // 16), torch.uint8, dev, stream),
                          _new_result(1, torch.float32, dev, stream))
    if workspace is None:
        workspace = _new(lib().nvfp4_quantize_workspace_size(), torch.uint8, dev, stream)
    _check(lib().nvfp4_quantize(x.data_ptr(), _dtype_code(x), rows, cols, _ptr(g), _ptr(out.g),
                                out.codes.data_ptr(), out.scales.data_ptr(), workspace.data_ptr(),
                                workspace.numel(), _stream(stream)))
    return out


# ------------------------------------------------------------------ packed weights
def nvfp4_weight_repack(codes, scales, out=None, stream=None):
    """Row-major NVFP4 weights codes uint8 [E, N, K/2], scales uint8 [E, N, K/16]
    -> packed tile layout (uint8 tensor) read by nvfp4_grouped_gemm(b_packed=...)."""
    import torch
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.uint8, "scales")
    E, N, K2 = codes.shape
    nbytes = lib().nvfp4_weight_packed_size(E, N, 2 * K2)
    if out is None:
        out = _new_result(nbytes, torch.uint8, codes.device, stream)
    _check(lib().nvfp4_weight_repack(codes.data_ptr(), scales.data_ptr(), E, N, 2 * K2, out.data_ptr(),
                                     out.numel(), _stream(stream)))
    return out


# ------------------------------------------------------------------ route + quantise
def moe_route_quantize(logits, k: int, x, g=None, out: Routing | None = None, xq: NVFP4Tensor | None = None,
                       workspace=None, stream=None) -> tuple[Routing, NVFP4Tensor]:
    """moe_route_permute(logits, k) and nvfp4_quantize(x, g) in one call whose
    kernels share launches; the outputs are those of the two calls."""
    import torch
    _need(logits, torch.float32, "logits")
    _need(x, x.dtype, "x")
    T, E = logits.shape
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, cols] with the logits' T rows")
    cols = x.shape[1]
    dev = logits.device
    if out is None:
        out = _new_routing(T, E, k, dev, stream)
    if xq is None:
        xq = NVFP4Tensor(_new_result((T, cols // 2), torch.uint8, dev, stream),
                         _new_result((T, cols // 16), torch.uint8, dev, stream),
                         _new_result(1, torch.float32, dev, stream))
    nbytes = lib().moe_route_quantize_workspace_size(T, E, k)
    if workspace is None:
        workspace = _new(max(nbytes, 16), torch.uint8, dev, stream)
    _check(lib().moe_route_quantize(
        logits.data_ptr(), T, E, k, out.topk_ids.data_ptr(), out.topk_w.data_ptr(), out.counts.data_ptr(),
        out.offsets.data_ptr(), out.perm_src_token.data_ptr(), out.perm_of_assignment.data_ptr(),
        _ptr(out.perm_weight), x.data_ptr(), _dtype_code(x), cols, _ptr(g), _ptr(xq.g), xq.codes.data_ptr(),
        xq.scales.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(stream)))
    return out, xq


def moe_route_quantize_noalloc(logits, k: int, x, out: Routing, xq: NVFP4Tensor, g=None, stream=None):
    """moe_route_quantize with the library's per-device scratch instead of a
    workspace: allocates nothing (outputs are the caller's ``out`` and ``xq``)."""
    import torch
    _need(logits, torch.float32, "logits")
    _need(x, x.dtype, "x")
    T, E = logits.shape
    if x.dim() != 2 or x.shape[0] != T:
        raise ValueError("x must be [T, cols] with the logits' T rows")
    cols = x.shape[1]
    if tuple(out.topk_ids.shape) != (T, k) or out.perm_src_token.numel() < T * k or out.offsets.numel() < E + 1:
        raise ValueError("routing outputs do not match T, E, k")
    if tuple(xq.codes.shape) != (T, cols // 2) or tuple(xq.scales.shape) != (T, cols // 16):
        raise ValueError("xq does not match x")
    _check(lib().moe_route_quantize_noalloc(
        logits.data_ptr(), T, E, k, out.topk_ids.data_ptr(), out.topk_w.data_ptr(), out.counts.data_ptr(),
        out.offsets.data_ptr(), out.perm_src_token.data_ptr(), out.perm_of_assignment.data_ptr(),
        _ptr(out.perm_weight), x.data_ptr(), _dtype_code(x), cols, _ptr(g), _ptr(xq.g), xq.codes.data_ptr(),
        xq.scales.data_ptr(), _stream(stream)))
    return out, xq


# ---------------------------------------------------------------------------- gemm
def nvfp4_grouped_gemm(a: NVFP4Tensor, b_codes, b_scales, b_g, offsets, *, m_total: int, a_rows=None,
                       epilogue: int = EPI_F32, out=None, out_rows: int = 0, out_codes=None,
                       out_scales=None, out_g=None, row_token=None, row_weight=None,
                       max_rows_per_expert_hint: int = 0, b_packed=None, stream=None):
    """Grouped NVFP4 GEMM (see include/nvfp4moe.h).  b_codes uint8 [E, N, K/2],
    b_scales uint8 [E, N, K/16], b_g float32 [E], offsets int32 [E+1] (device).
    With b_packed (from nvfp4_weight_repack), b_codes/b_scales give only the
    shapes (they may be meta or empty-strided tensors) and are not read."""
    import torch
    E, N, K2 = b_codes.shape
    K = 2 * K2
    _need(a.codes, torch.uint8, "a.codes")
    _need(a.scales, torch.uint8, "a.scales")
    if b_packed is None:
        _need(b_codes, torch.uint8, "b_codes")
        _need(b_scales, torch.uint8, "b_scales")
    else:
        _need(b_packed, torch.uint8, "b_packed")
        if b_packed.numel() < lib().nvfp4_weight_packed_size(E, N, K):
            raise ValueError("b_packed is smaller than the packed size of [E, N, K]")
    _need(b_g, torch.float32, "b_g")
    _need(offsets, torch.int32, "offsets")
    if a.codes.shape[1] != K2 or tuple(b_scales.shape) != (E, N, K // 16):
        raise ValueError("operand shapes disagree")
    a_rows_total = a.codes.shape[0]
    if tuple(a.scales.shape) != (a_rows_total, K // 16):
        raise ValueError(f"a.scales: expected [{a_rows_total}, {K // 16}], got {list(a.scales.shape)}")
    if a.g.numel() < 1 or b_g.numel() < E:
        raise ValueError("a.g needs 1 and b_g needs E float32 values")
    if offsets.numel() < E + 1:
        raise ValueError(f"offsets: {offsets.numel()} values, expected E+1 = {E + 1}")
    if a_rows is not None:
        _need(a_rows, torch.int32, "a_rows")
        if a_rows.numel() < m_total:
            raise ValueError(f"a_rows: {a_rows.numel()} values, expected m_total = {m_total}")
    dev = b_codes.device
    I = N // 2
    if epilogue in (EPI_F32, EPI_BF16):
        want = torch.float32 if epilogue == EPI_F32 else torch.bfloat16
        if out is None:
            out = _new_result((m_total, N), want, dev, stream)
        else:
            _need(out, want, "out")
            if tuple(out.shape) != (m_total, N):
                raise ValueError(f"out: expected [{m_total}, {N}], got {list(out.shape)}")
    if epilogue == EPI_SWIGLU_NVFP4:
        if out_g is None:
            raise ValueError("EPI_SWIGLU_NVFP4 needs out_g (the per-tensor scale of h)")
        _need(out_g, torch.float32, "out_g")
        if out_codes is None:
            out_codes = _new_result((m_total, I // 2), torch.uint8, dev, stream)
            out_scales = _new_result((m_total, I // 16), torch.uint8, dev, stream)
        _need(out_codes, torch.uint8, "out_codes")
        _need(out_scales, torch.uint8, "out_scales")
        if tuple(out_codes.shape) != (m_total, I // 2) or tuple(out_scales.shape) != (m_total, I // 16):
            raise ValueError(f"out_codes/out_scales: expected [{m_total}, {I // 2}] and [{m_total}, {I // 16}]")
    if epilogue == EPI_COMBINE_F32:
        if out is None or row_token is None or row_weight is None:
            raise ValueError("EPI_COMBINE_F32 needs out, row_token and row_weight")
        _need(out, torch.float32, "out")
        _need(row_token, torch.int32, "row_token")
        _need(row_weight, torch.float32, "row_weight")
        if tuple(out.shape) != (out_rows, N) or row_token.numel() < m_total or row_weight.numel() < m_total:
            raise ValueError(f"combine epilogue: out must be [out_rows={out_rows}, {N}], row_token and row_weight "
                             f"at least m_total = {m_total} long")
    args = GemmArgs(
        a_codes=a.codes.data_ptr(), a_scales=a.scales.data_ptr(), a_g=a.g.data_ptr(), a_rows=_ptr(a_rows),
        a_rows_total=a_rows_total,
        b_codes=None if b_packed is not None else b_codes.data_ptr(),
        b_scales=None if b_packed is not None else b_scales.data_ptr(), b_packed=_ptr(b_packed),
        b_g=b_g.data_ptr(), offsets=offsets.data_ptr(), E=E, N=N, K=K, m_total=m_total, epilogue=epilogue,
        out=_ptr(out), out_rows=out_rows, out_codes=_ptr(out_codes), out_scales=_ptr(out_scales),
        out_g=_ptr(out_g), row_token=_ptr(row_token), row_weight=_ptr(row_weight),
        max_rows_per_expert_hint=max_rows_per_expert_hint)
    _check(lib().nvfp4_grouped_gemm(ctypes.byref(args), _stream(stream)))
    if epilogue == EPI_SWIGLU_NVFP4:
        return NVFP4Tensor(out_codes, out_scales, out_g)
    return out


# ---------------------------------------------------------------------- expert FFN
def moe_expert_ffn_workspace(E: int, m_total: int, H: int, I: int, device):
    import torch
    n = lib().moe_expert_ffn_workspace_size(E, m_total, H, I)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def moe_expert_ffn(xq: NVFP4Tensor, perm_src_token, offsets, w_gu_packed, g_gu, w_dn_packed, g_dn, g_h, *, H: int,
                   I: int, m_total: int, h: NVFP4Tensor | None = None, y=None, workspace=None,
                   max_rows_per_expert_hint: int = 0, perm_of_assignment=None, topk_w=None, k: int = 0, out=None,
                   stream=None):
    """gate_up + SwiGLU/requant + down for all experts (see include/nvfp4moe.h):
    returns (h NVFP4Tensor [m_total, I], y bf16 [m_total, H]); with
    perm_of_assignment, topk_w ([T, k]) and k also the weighted top-k combine
    out bf16 [T, H] (fused into the launch in the one-launch regime), returned
    as a third element."""
    import torch
    E = offsets.numel() - 1
    dev = offsets.device
    _need(xq.codes, torch.uint8, "x codes")
    _need(xq.scales, torch.uint8, "x scales")
    if tuple(xq.codes.shape[1:]) != (H // 2,) or tuple(xq.scales.shape) != (xq.codes.shape[0], H // 16):
        raise ValueError("x codes/scales do not match H")
    _need(perm_src_token, torch.int32, "perm_src_token")
    _need(offsets, torch.int32, "offsets")
    if perm_src_token.numel() < m_total:
        raise ValueError("perm_src_token shorter than m_total")
    for t, name, n in ((w_gu_packed, "w_gu_packed", lib().nvfp4_weight_packed_size(E, 2 * I, H)),
                       (w_dn_packed, "w_dn_packed", lib().nvfp4_weight_packed_size(E, H, I))):
        _need(t, torch.uint8, name)
        if t.numel() < n:
            raise ValueError(f"{name}: {t.numel()} bytes, the packed size is {n}")
    for t, name, n in ((g_gu, "g_gu", E), (g_dn, "g_dn", E), (g_h, "g_h", 1)):
        _need(t, torch.float32, name)
        if t.numel() < n:
            raise ValueError(f"{name}: needs {n} values")
    if h is None:
        h = NVFP4Tensor(_new_result((m_total, I // 2), torch.uint8, dev, stream),
                        _new_result((m_total, I // 16), torch.uint8, dev, stream), g_h)
    if tuple(h.codes.shape) != (m_total, I // 2) or tuple(h.scales.shape) != (m_total, I // 16):
        raise ValueError("h codes/scales must be [m_total, I/2] and [m_total, I/16]")
    if y is None:
        y = _new_result((m_total, H), torch.bfloat16, dev, stream)
    _need(y, torch.bfloat16, "y")
    if tuple(y.shape) != (m_total, H):
        raise ValueError("y must be bf16 [m_total, H]")
    T = 0
    if perm_of_assignment is not None:
        if topk_w is None or k <= 0 or m_total % k:
            raise ValueError("the combine needs topk_w and k > 0 dividing m_total")
        T = m_total // k
        _need(perm_of_assignment, torch.int32, "perm_of_assignment")
        _need(topk_w, torch.float32, "topk_w")
        if perm_of_assignment.numel() < m_total or topk_w.numel() < m_total:
            raise ValueError("perm_of_assignment and topk_w need T * k values")
        if out is None:
            out = _new_result((T, H), torch.bfloat16, dev, stream)
        _need(out, torch.bfloat16, "out")
        if tuple(out.shape) != (T, H):
            raise ValueError("out must be bf16 [T, H]")
    if workspace is None:
        workspace = _new(max(lib().moe_expert_ffn_workspace_size(E, m_total, H, I), 256), torch.uint8, dev, stream)
    args = FfnArgs(x_codes=xq.codes.data_ptr(), x_scales=xq.scales.data_ptr(), x_g=xq.g.data_ptr(),
                   x_rows=xq.codes.shape[0], perm_src_token=perm_src_token.data_ptr(), offsets=offsets.data_ptr(),
                   E=E, H=H, I=I, m_total=m_total, w_gu_packed=w_gu_packed.data_ptr(), g_gu=g_gu.data_ptr(),
                   w_dn_packed=w_dn_packed.data_ptr(), g_dn=g_dn.data_ptr(), g_h=g_h.data_ptr(),
                   h_codes=h.codes.data_ptr(), h_scales=h.scales.data_ptr(), y=y.data_ptr(),
                   max_rows_per_expert_hint=max_rows_per_expert_hint,
                   out=out.data_ptr() if T else None,
                   perm_of_assignment=perm_of_assignment.data_ptr() if T else None,
                   topk_w=topk_w.data_ptr() if T else None, T=T, k=k if T else 0)
    _check(lib().moe_expert_ffn(ctypes.byref(args), workspace.data_ptr(), workspace.numel(), _stream(stream)))
    if T:
        return NVFP4Tensor(h.codes, h.scales, g_h), y, out
    return NVFP4Tensor(h.codes, h.scales, g_h), y


# --------------------------------------------------------------------------- MXFP4
@dataclass
class MXFP4Tensor:
    codes: "object"     # uint8 [rows, cols/2]
    scales: "object"    # uint8 [rows, cols/32], E8M0


def mxfp4_quantize(x, out: MXFP4Tensor | None = None, stream=None) -> MXFP4Tensor:
    """x bf16/float32 [rows, cols] (or [..., cols]) -> MXFP4Tensor (E8M0 scale per 32 values)."""
    import torch
    _need(x, x.dtype, "x")
    cols = x.shape[-1]
    rows = x.numel() // cols
    dev = x.device
    if out is None:
        out = MXFP4Tensor(_new_result(x.shape[:-1] + (cols // 2,), torch.uint8, dev, stream),
                          _new_result(x.shape[:-1] + (cols // 32,), torch.uint8, dev, stream))
    if out.codes.numel() != rows * (cols // 2) or out.scales.numel() != rows * (cols // 32):
        raise ValueError("out codes/scales do not match x")
    _need(out.codes, torch.uint8, "out.codes")
    _need(out.scales, torch.uint8, "out.scales")
    _check(lib().mxfp4_quantize(x.data_ptr(), _dtype_code(x), rows, cols, out.codes.data_ptr(), out.scales.data_ptr(),
                                _stream(stream)))
    return out


def mxfp4_weight_repack(b: MXFP4Tensor, out=None, stream=None):
    """MXFP4 weights codes [E, N, K/2], scales [E, N, K/32] -> packed tiles
    (uint8 tensor) for mxfp4_grouped_gemm(b_packed=...)."""
    import torch
    _need(b.codes, torch.uint8, "codes")
    _need(b.scales, torch.uint8, "scales")
    E, N, K2 = b.codes.shape
    nbytes = lib().mxfp4_weight_packed_size(E, N, 2 * K2)
    if out is None:
        out = _new_result(nbytes, torch.uint8, b.codes.device, stream)
    _check(lib().mxfp4_weight_repack(b.codes.data_ptr(), b.scales.data_ptr(), E, N, 2 * K2, out.data_ptr(),
                                     out.numel(), _stream(stream)))
    return out


def _new_ones(n, dev, stream):
    """n float32 ones, filled on the call's own stream."""
    import torch
    with torch.cuda.stream(stream):        # None: no change
        return torch.ones(n, dtype=torch.float32, device=dev)


def mxfp4_grouped_gemm(a: MXFP4Tensor, b: MXFP4Tensor, offsets, *, m_total: int, a_rows=None, epilogue: int = EPI_F32,
                       out=None, out_codes=None, out_scales=None, a_g=None, b_g=None,
                       max_rows_per_expert_hint: int = 0, b_packed=None, stream=None):
    """Grouped MXFP4 GEMM (see include/nvfp4moe.h): a [rows, K], b [E, N, K]
    (codes/scales), offsets int32 [E+1].  Epilogues F32, BF16, or
    EPI_SWIGLU_NVFP4 read as SwiGLU + MXFP4 requantisation (returns an
    MXFP4Tensor of h).  a_g / b_g: optional float32 multipliers (1 / E values)."""
    import torch
    E, N, K2 = b.codes.shape
    K = 2 * K2
    dev = b.codes.device
    for t, name in ((a.codes, "a.codes"), (a.scales, "a.scales")):
        _need(t, torch.uint8, name)
    if b_packed is None:
        _need(b.codes, torch.uint8, "b.codes")
        _need(b.scales, torch.uint8, "b.scales")
    else:
        _need(b_packed, torch.uint8, "b_packed")
        if b_packed.numel() < lib().mxfp4_weight_packed_size(E, N, K):
            raise ValueError("b_packed is smaller than the packed size of [E, N, K]")
    _need(offsets, torch.int32, "offsets")
    rows_a = a.codes.shape[0]
    if tuple(a.codes.shape) != (rows_a, K2) or tuple(a.scales.shape) != (rows_a, K // 32) \
            or tuple(b.scales.shape) != (E, N, K // 32):
        raise ValueError("operand shapes disagree")
    if offsets.numel() < E + 1:
        raise ValueError("offsets needs E+1 values")
    if a_rows is not None:
        _need(a_rows, torch.int32, "a_rows")
        if a_rows.numel() < m_total:
            raise ValueError("a_rows shorter than m_total")
    if a_g is None:
        a_g = _new_ones(1, dev, stream)
    if b_g is None:
        b_g = _new_ones(E, dev, stream)
    _need(a_g, torch.float32, "a_g")
    _need(b_g, torch.float32, "b_g")
    I = N // 2
    if epilogue in (EPI_F32, EPI_BF16):
        want = torch.float32 if epilogue == EPI_F32 else torch.bfloat16
        if out is None:
            out = _new_result((m_total, N), want, dev, stream)
        _need(out, want, "out")
        if tuple(out.shape) != (m_total, N):
            raise ValueError("out must be [m_total, N]")
    elif epilogue == EPI_SWIGLU_NVFP4:
        if out_codes is None:
            out_codes = _new_result((m_total, I // 2), torch.uint8, dev, stream)
            out_scales = _new_result((m_total, I // 32), torch.uint8, dev, stream)
        if tuple(out_codes.shape) != (m_total, I // 2) or tuple(out_scales.shape) != (m_total, I // 32):
            raise ValueError("out_codes/out_scales must be [m_total, I/2] and [m_total, I/32]")
    args = GemmArgs(a_codes=a.codes.data_ptr(), a_scales=a.scales.data_ptr(), a_g=a_g.data_ptr(), a_rows=_ptr(a_rows),
                    a_rows_total=rows_a, b_codes=None if b_packed is not None else b.codes.data_ptr(),
                    b_scales=None if b_packed is not None else b.scales.data_ptr(), b_packed=_ptr(b_packed),
                    b_g=b_g.data_ptr(), offsets=offsets.data_ptr(), E=E, N=N, K=K, m_total=m_total,
                    epilogue=epilogue, out=_ptr(out), out_rows=0, out_codes=_ptr(out_codes),
                    out_scales=_ptr(out_scales), out_g=None, row_token=None, row_weight=None,
                    max_rows_per_expert_hint=max_rows_per_expert_hint)
    _check(lib().mxfp4_grouped_gemm(ctypes.byref(args), _stream(stream)))
    if epilogue == EPI_SWIGLU_NVFP4:
        return MXFP4Tensor(out_codes, out_scales)
    return out


# --------------------------------------------------------------------------- FP8
FP8_BLOCK = 128


@dataclass
class FP8Tensor:
    codes: "object"     # uint8 [..., rows, cols], E4M3 bytes
    scales: "object"    # float32 [..., ceil(rows/block_rows), cols/128]
    block_rows: int     # 1 (activations) or 128 (weights)


def fp8_quantize(x, block_rows: int = 1, out: FP8Tensor | None = None, stream=None) -> FP8Tensor:
    """x bf16/float32 [rows, cols] (block_rows 1) or [batch, rows, cols]
    (block_rows 128: one scale per 128 x 128 tile of each matrix) -> FP8Tensor."""
    import torch
    _need(x, x.dtype, "x")
    cols = x.shape[-1]
    if block_rows == 1:
        batch, rows = 1, x.numel() // cols
        sshape = x.shape[:-1] + (cols // FP8_BLOCK,)
    else:
        rows = x.shape[-2]
        batch = x.numel() // (rows * cols)
        sshape = x.shape[:-2] + ((rows + FP8_BLOCK - 1) // FP8_BLOCK, cols // FP8_BLOCK)
    dev = x.device
    if out is None:
        out = FP8Tensor(_new_result(x.shape, torch.uint8, dev, stream),
                        _new_result(sshape, torch.float32, dev, stream), block_rows)
    if out.codes.numel() != x.numel() or tuple(out.scales.shape) != tuple(sshape):
        raise ValueError("out codes/scales do not match x")
    _need(out.codes, torch.uint8, "out.codes")
    _need(out.scales, torch.float32, "out.scales")
    _check(lib().fp8_quantize(x.data_ptr(), _dtype_code(x), batch, rows, cols, block_rows, out.codes.data_ptr(),
                              out.scales.data_ptr(), _stream(stream)))
    return out


def fp8_swiglu_quantize(gate_up, out: FP8Tensor | None = None, stream=None) -> FP8Tensor:
    """gate_up float32/bf16 [M, 2I] -> FP8 h = silu(gate) * up with 1 x 128 blocks."""
    import torch
    _need(gate_up, gate_up.dtype, "gate_up")
    M, N2 = gate_up.shape
    I = N2 // 2
    dev = gate_up.device
    if out is None:
        out = FP8Tensor(_new_result((M, I), torch.uint8, dev, stream),
                        _new_result((M, I // FP8_BLOCK), torch.float32, dev, stream), 1)
    if tuple(out.codes.shape) != (M, I) or tuple(out.scales.shape) != (M, I // FP8_BLOCK):
        raise ValueError("out codes/scales must be [M, I] and [M, I/128]")
    _need(out.codes, torch.uint8, "out.codes")
    _need(out.scales, torch.float32, "out.scales")
    _check(lib().fp8_swiglu_quantize(gate_up.data_ptr(), _dtype_code(gate_up), M, I, out.codes.data_ptr(),
                                     out.scales.data_ptr(), _stream(stream)))
    return out


def fp8_weight_repack(codes, out=None, stream=None):
    """FP8 weight codes [E, N, K] -> packed tiles (uint8 tensor) for fp8_grouped_gemm."""
    import torch
    _need(codes, torch.uint8, "codes")
    E, N, K = codes.shape
    nbytes = lib().fp8_weight_packed_size(E, N, K)
    if out is None:
        out = _new_result(nbytes, torch.uint8, codes.device, stream)
    _check(lib().fp8_weight_repack(codes.data_ptr(), E, N, K, out.data_ptr(), out.numel(), _stream(stream)))
    return out


def fp8_grouped_gemm(a: FP8Tensor, b_packed, b_scales, offsets, *, N: int, m_total: int, a_rows=None,
                     epilogue: int = EPI_F32, out=None, max_rows_per_expert_hint: int = 0, stream=None):
    """Grouped FP8 GEMM (see include/nvfp4moe.h): a [rows, K] (1 x 128 blocks),
    b_packed from fp8_weight_repack, b_scales float32 [E, ceil(N/128), K/128],
    offsets int32 [E+1].  Epilogues F32 or BF16 (returns out), or
    EPI_SWIGLU_NVFP4 read as SwiGLU + FP8 requant of h (N = 2I, I % 128 == 0;
    out: an FP8Tensor for h or None; returns it)."""
    import torch
    rows_a, K = a.codes.shape
    E = b_scales.shape[0]
    dev = a.codes.device
    if a.block_rows != 1:
        raise ValueError("A must be quantised with 1 x 128 blocks")
    _need(a.codes, torch.uint8, "a.codes")
    _need(a.scales, torch.float32, "a.scales")
    _need(b_packed, torch.uint8, "b_packed")
    _need(b_scales, torch.float32, "b_scales")
    _need(offsets, torch.int32, "offsets")
    if tuple(a.scales.shape) != (rows_a, K // FP8_BLOCK) or \
            tuple(b_scales.shape) != (E, (N + FP8_BLOCK - 1) // FP8_BLOCK, K // FP8_BLOCK):
        raise ValueError("operand shapes disagree")
    if b_packed.numel() < lib().fp8_weight_packed_size(E, N, K):
        raise ValueError("b_packed is smaller than the packed size of [E, N, K]")
    if offsets.numel() < E + 1:
        raise ValueError("offsets needs E+1 values")
    if a_rows is not None:
        _need(a_rows, torch.int32, "a_rows")
        if a_rows.numel() < m_total:
            raise ValueError("a_rows shorter than m_total")
    if epilogue == EPI_SWIGLU_NVFP4:
        if N % (2 * FP8_BLOCK) != 0:
            raise ValueError("fp8_grouped_gemm: SwiGLU needs N = 2I with I % 128 == 0")
        I = N // 2
        if out is None:
            out = FP8Tensor(_new_result((m_total, I), torch.uint8, dev, stream),
                            _new_result((m_total, I // FP8_BLOCK), torch.float32, dev, stream), 1)
        _need(out.codes, torch.uint8, "out.codes")
        _need(out.scales, torch.float32, "out.scales")
        if tuple(out.codes.shape) != (m_total, I) or tuple(out.scales.shape) != (m_total, I // FP8_BLOCK):
            raise ValueError("out codes/scales must be [m_total, I] and [m_total, I/128]")
        args = Fp8GemmArgs(a_codes=a.codes.data_ptr(), a_scales=a.scales.data_ptr(), a_rows=_ptr(a_rows),
                           a_rows_total=rows_a, b_packed=b_packed.data_ptr(), b_scales=b_scales.data_ptr(),
                           offsets=offsets.data_ptr(), E=E, N=N, K=K, m_total=m_total, epilogue=epilogue, out=None,
                           max_rows_per_expert_hint=max_rows_per_expert_hint, out_codes=out.codes.data_ptr(),
                           out_scales=out.scales.data_ptr())
        _check(lib().fp8_grouped_gemm(ctypes.byref(args), _stream(stream)))
        return out
    if epilogue not in (EPI_F32, EPI_BF16):
        raise ValueError("fp8_grouped_gemm: epilogue F32, BF16 or SwiGLU")
    want = torch.float32 if epilogue == EPI_F32 else torch.bfloat16
    if out is None:
        out = _new_result((m_total, N), want, dev, stream)
    _need(out, want, "out")
    if tuple(out.shape) != (m_total, N):
        raise ValueError("out must be [m_total, N]")
    args = Fp8GemmArgs(a_codes=a.codes.data_ptr(), a_scales=a.scales.data_ptr(), a_rows=_ptr(a_rows),
                       a_rows_total=rows_a, b_packed=b_packed.data_ptr(), b_scales=b_scales.data_ptr(),
                       offsets=offsets.data_ptr(), E=E, N=N, K=K, m_total=m_total, epilogue=epilogue,
                       out=out.data_ptr(), max_rows_per_expert_hint=max_rows_per_expert_hint)
    _check(lib().fp8_grouped_gemm(ctypes.byref(args), _stream(stream)))
    return out


# ----------------------------------------------------------------- 16-bit expert FFN
def _dtype16(t, name):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float16:
        return F16
    raise TypeError(f"{name}: expected bfloat16 or float16, got {t.dtype}")


def _rows_of(a_rows, source, m_total, dev, name):
    """Checks of a gathered (a_rows given) or direct row operand."""
    import torch
    if m_total < 0:
        raise ValueError("m_total must be >= 0")
    if a_rows is not None:
        _need(a_rows, torch.int32, "a_rows", dev)
        if a_rows.numel() < m_total:
            raise ValueError(f"a_rows: {a_rows.numel()} values, expected m_total = {m_total}")
    elif source.shape[0] < m_total:
        raise ValueError(f"{name}: {source.shape[0]} rows, expected m_total = {m_total}")


def _group(b, offsets, dev):
    """E of weights [E, ...] with their offsets."""
    import torch
    _need(offsets, torch.int32, "offsets", dev)
    E = b.shape[0]
    if offsets.numel() < E + 1:
        raise ValueError(f"offsets: {offsets.numel()} values, expected E+1 = {E + 1}")
    return E


def _result(out, shape, dtype, like, name, stream):
    """A given result checked, or a new one on ``like``'s device."""
    if out is None:
        if stream is None:
            return _empty(shape, dtype, like.device)
        return _new_result(shape, dtype, like.device, stream)
    _need(out, dtype, name, like.device)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {list(shape)}, got {list(out.shape)}")
    return out


def _scratch(workspace, need, dev, stream):
    import torch
    if workspace is None:
        return _new(max(need, 256), torch.uint8, dev, stream)
    _need(workspace, torch.uint8, "workspace", dev)
    return workspace


def moe_gated_ffn(x, w, offsets, *, m_total: int, a_rows=None, activation: int = ACT_SILU, save_gu: bool = False,
                  out=None, gu=None, max_rows_per_expert_hint: int = 0, stream=None):
    """h = act(x Wg^T) * (x Wu^T) per expert (see include/nvfp4moe.h): x bf16/f16
    [rows, H], w [E, 2I, H] (rows [0, I) gate), offsets int32 [E+1] -> h
    [m_total, I].  save_gu (or a float32 gu [m_total, 2I]): returns (h, gu) with
    the pre-activations that moe_gated_ffn_backward reads."""
    import torch
    if x.dim() != 2 or w.dim() != 3:
        raise ValueError("x must be [rows, H] and w [E, 2I, H]")
    dev = w.device
    code = _dtype16(w, "w")
    _need(w, w.dtype, "w", dev)
    _need(x, w.dtype, "x", dev)
    E = _group(w, offsets, dev)
    H, I = w.shape[2], w.shape[1] // 2
    if x.shape[1] != H or w.shape[1] != 2 * I:
        raise ValueError("operand shapes disagree")
    _rows_of(a_rows, x, m_total, dev, "x")
    h = _result(out, (m_total, I), w.dtype, w, "out", stream)
    if save_gu or gu is not None:
        gu = _result(gu, (m_total, 2 * I), torch.float32, w, "gu", stream)
    args = GatedArgs(x=x.data_ptr(), dtype=code, a_rows=_ptr(a_rows), x_rows=x.shape[0], w=w.data_ptr(),
                     offsets=offsets.data_ptr(), E=E, H=H, I=I, m_total=m_total, activation=activation,
                     max_rows_per_expert_hint=max_rows_per_expert_hint, h=h.data_ptr(), gu=_ptr(gu))
    _call(dev, stream, lib().moe_gated_ffn, ctypes.byref(args))
    return h if gu is None else (h, gu)


def moe_gated_ffn_backward(dh, gu, x, w, offsets, *, a_rows=None, activation: int = ACT_SILU, need_dx: bool = True,
                           need_dw: bool = True, dx=None, dw=None, workspace=None, max_rows_per_expert_hint: int = 0,
                           stream=None):
    """Gradients of moe_gated_ffn: dh [m_total, I], gu as saved -> (dx
    [m_total, H] one row per GEMM row, dw [E, 2I, H]); None where not needed.
    For gathered x the gradient of the tokens is
    moe_unpermute_combine(dx, perm_of_assignment, None, T, k)."""
    import torch
    if x.dim() != 2 or w.dim() != 3 or dh.dim() != 2:
        raise ValueError("x must be [rows, H], w [E, 2I, H] and dh [m_total, I]")
    if not (need_dx or need_dw):
        raise ValueError("neither dx nor dw is needed")
    dev = w.device
    code = _dtype16(w, "w")
    _need(w, w.dtype, "w", dev)
    _need(x, w.dtype, "x", dev)
    _need(dh, w.dtype, "dh", dev)
    _need(gu, torch.float32, "gu", dev)
    E = _group(w, offsets, dev)
    H, I, m_total = w.shape[2], w.shape[1] // 2, dh.shape[0]
    if x.shape[1] != H or w.shape[1] != 2 * I or dh.shape[1] != I or tuple(gu.shape) != (m_total, 2 * I):
        raise ValueError("operand shapes disagree")
    _rows_of(a_rows, x, m_total, dev, "x")
    dx = _result(dx, (m_total, H), w.dtype, w, "dx", stream) if need_dx else None
    dw = _result(dw, w.shape, w.dtype, w, "dw", stream) if need_dw else None
    if m_total == 0 and not need_dw:
        return dx, dw
    ws = _scratch(workspace, lib().moe_gated_ffn_backward_workspace_size(E, H, I, m_total), dev, stream)
    args = GatedGradArgs(x=x.data_ptr(), dtype=code, a_rows=_ptr(a_rows), x_rows=x.shape[0], w=w.data_ptr(),
                         offsets=offsets.data_ptr(), E=E, H=H, I=I, m_total=m_total, activation=activation,
                         max_rows_per_expert_hint=max_rows_per_expert_hint, gu=gu.data_ptr(), dh=dh.data_ptr(),
                         dx=_ptr(dx), dw=_ptr(dw))
    _call(dev, stream, lib().moe_gated_ffn_backward, ctypes.byref(args), ws.data_ptr(), ws.numel())
    return dx, dw


def moe_grouped_gemm(a, b, offsets, *, m_total: int, a_rows=None, out=None, out_dtype=None,
                     max_rows_per_expert_hint: int = 0, stream=None):
    """y[p] = a[r] b[e]^T per expert (see include/nvfp4moe.h): a bf16/f16 [rows, K],
    b [E, N, K], offsets int32 [E+1] -> [m_total, N] in a's dtype or float32."""
    import torch
    if a.dim() != 2 or b.dim() != 3:
        raise ValueError("a must be [rows, K] and b [E, N, K]")
    dev = b.device
    code = _dtype16(b, "b")
    _need(b, b.dtype, "b", dev)
    _need(a, b.dtype, "a", dev)
    E = _group(b, offsets, dev)
    N, K = b.shape[1], b.shape[2]
    if a.shape[1] != K:
        raise ValueError("operand shapes disagree")
    _rows_of(a_rows, a, m_total, dev, "a")
    want = out.dtype if out is not None and out_dtype is None else (out_dtype or b.dtype)
    if want not in (b.dtype, torch.float32):
        raise TypeError(f"out: {b.dtype} or float32, got {want}")
    out = _result(out, (m_total, N), want, b, "out", stream)
    args = ProductArgs(a=a.data_ptr(), dtype=code, a_rows=_ptr(a_rows), a_rows_total=a.shape[0], b=b.data_ptr(),
                       offsets=offsets.data_ptr(), E=E, N=N, K=K, m_total=m_total,
                       out_dtype=F32 if want == torch.float32 else code,
                       max_rows_per_expert_hint=max_rows_per_expert_hint, out=out.data_ptr())
    _call(dev, stream, lib().moe_grouped_gemm, ctypes.byref(args))
    return out


def moe_grouped_gemm_backward(dy, a, b, offsets, *, a_rows=None, need_da: bool = True, need_db: bool = True, da=None,
                              db=None, workspace=None, max_rows_per_expert_hint: int = 0, stream=None):
    """Gradients of moe_grouped_gemm: dy [m_total, N] in b's dtype -> (da
    [m_total, K] one row per GEMM row, db [E, N, K]); None where not needed."""
    if a.dim() != 2 or b.dim() != 3 or dy.dim() != 2:
        raise ValueError("a must be [rows, K], b [E, N, K] and dy [m_total, N]")
    if not (need_da or need_db):
        raise ValueError("neither da nor db is needed")
    dev = b.device
    code = _dtype16(b, "b")
    _need(b, b.dtype, "b", dev)
    _need(a, b.dtype, "a", dev)
    _need(dy, b.dtype, "dy", dev)
    E = _group(b, offsets, dev)
    N, K, m_total = b.shape[1], b.shape[2], dy.shape[0]
    if a.shape[1] != K or dy.shape[1] != N:
        raise ValueError("operand shapes disagree")
    _rows_of(a_rows, a, m_total, dev, "a")
    da = _result(da, (m_total, K), b.dtype, b, "da", stream) if need_da else None
    db = _result(db, b.shape, b.dtype, b, "db", stream) if need_db else None
    if m_total == 0 and not need_db:
        return da, db
    need = lib().moe_grouped_gemm_backward_workspace_size(E, N, K, m_total)
    ws = _scratch(workspace, need, dev, stream) if need else None
    args = ProductGradArgs(a=a.data_ptr(), dtype=code, a_rows=_ptr(a_rows), a_rows_total=a.shape[0], b=b.data_ptr(),
                           offsets=offsets.data_ptr(), E=E, N=N, K=K, m_total=m_total,
                           max_rows_per_expert_hint=max_rows_per_expert_hint, dy=dy.data_ptr(), da=_ptr(da),
                           db=_ptr(db))
    _call(dev, stream, lib().moe_grouped_gemm_backward, ctypes.byref(args), _ptr(ws), ws.numel() if need else 0)
    return da, db


# --------------------------------------------------------------------------- INT8
@dataclass
class INT8Tensor:
    codes: "object"     # int8 [..., rows, cols]
    scales: "object"    # float32 [..., rows]


def int8_quantize(x, out: INT8Tensor | None = None, stream=None) -> INT8Tensor:
    """x bf16/float32 [..., rows, cols] -> INT8Tensor with one scale per row
    (tokens of activations, output channels of weights)."""
    import torch
    code = _dtype_code(x)
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("x must have at least one dimension and one column")
    dev = x.device
    _need(x, x.dtype, "x", dev)
    cols = x.shape[-1]
    if out is None:
        out = INT8Tensor(_result(None, x.shape, torch.int8, x, "out.codes", stream),
                         _result(None, x.shape[:-1], torch.float32, x, "out.scales", stream))
    else:
        _need(out.codes, torch.int8, "out.codes", dev)
        _need(out.scales, torch.float32, "out.scales", dev)
        if out.codes.shape != x.shape or out.scales.shape != x.shape[:-1]:
            raise ValueError("out codes/scales do not match x")
    if x.numel() == 0:
        return out
    _call(dev, stream, lib().int8_quantize, x.data_ptr(), code, x.numel() // cols, cols, out.codes.data_ptr(),
          out.scales.data_ptr())
    return out


def int8_grouped_gemm(a: INT8Tensor, b: INT8Tensor, offsets, *, m_total: int, a_rows=None, epilogue: int = EPI_BF16,
                      out=None, max_rows_per_expert_hint: int = 0, stream=None):
    """Grouped INT8 GEMM (see include/nvfp4moe.h): a [rows, K], b [E, N, K] with
    scales [E, N], offsets int32 [E+1].  Epilogues F32, BF16, or EPI_SWIGLU_BF16
    (N = 2I: returns bf16 h [m_total, I])."""
    import torch
    if a.codes.dim() != 2 or b.codes.dim() != 3:
        raise ValueError("a must be [rows, K] and b [E, N, K]")
    dev = b.codes.device
    _need(b.codes, torch.int8, "b.codes", dev)
    _need(b.scales, torch.float32, "b.scales", dev)
    _need(a.codes, torch.int8, "a.codes", dev)
    _need(a.scales, torch.float32, "a.scales", dev)
    E = _group(b.codes, offsets, dev)
    N, K = b.codes.shape[1], b.codes.shape[2]
    if a.codes.shape[1] != K or tuple(b.scales.shape) != (E, N) or tuple(a.scales.shape) != (a.codes.shape[0],):
        raise ValueError("operand shapes disagree")
    _rows_of(a_rows, a.codes, m_total, dev, "a")
    if epilogue not in (EPI_F32, EPI_BF16, EPI_SWIGLU_BF16):
        raise ValueError("int8_grouped_gemm: epilogue F32, BF16 or SWIGLU_BF16")
    out = _result(out, (m_total, N // 2 if epilogue == EPI_SWIGLU_BF16 else N),
                  torch.float32 if epilogue == EPI_F32 else torch.bfloat16, b.codes, "out", stream)
    args = Int8GemmArgs(a_codes=a.codes.data_ptr(), a_scales=a.scales.data_ptr(), a_rows=_ptr(a_rows),
                        a_rows_total=a.codes.shape[0], b_codes=b.codes.data_ptr(), b_scales=b.scales.data_ptr(),
                        offsets=offsets.data_ptr(), E=E, N=N, K=K, m_total=m_total, epilogue=epilogue,
                        max_rows_per_expert_hint=max_rows_per_expert_hint, out=out.data_ptr())
    _call(dev, stream, lib().int8_grouped_gemm, ctypes.byref(args))
    return out


# --------------------------------------------------------------------------- INT4
@dataclass
class INT4Tensor:
    codes: "object"     # uint8 [..., rows, cols/2]
    scales: "object"    # bf16/f16 [..., rows, cols/group]
    zeros: "object"     # uint8 [..., rows, cols/group] or None (8 everywhere)
    group: int          # 32, 64 or 128


def _need_int4(q, name, dev):
    """Checks of an INT4Tensor on ``dev``: the code of its scales' type."""
    import torch
    code = _dtype16(q.scales, name + ".scales")
    if q.group not in (32, 64, 128):
        raise ValueError(f"{name}: group {q.group} (32, 64 or 128)")
    _need(q.codes, torch.uint8, name + ".codes", dev)
    *lead, half = q.codes.shape
    if 2 * half % q.group:
        raise ValueError(f"{name}: {2 * half} columns, not a multiple of the group of {q.group}")
    shape = (*lead, 2 * half // q.group)
    _need_shape(q.scales, shape, q.scales.dtype, name + ".scales", dev)
    if q.zeros is not None:
        _need_shape(q.zeros, shape, torch.uint8, name + ".zeros", dev)
    return code


def int4_quantize(x, group: int = 128, zeros: bool = False, scale_dtype=None, out: INT4Tensor | None = None,
                  stream=None) -> INT4Tensor:
    """x float32/bf16/f16 [..., rows, cols] -> INT4Tensor, groups along the last
    axis; scales in x's 16-bit type, or scale_dtype (bf16 for float32 x)."""
    import torch
    code = _dtype_any(x, "x")
    dev = x.device
    _need(x, x.dtype, "x", dev)
    if group not in (32, 64, 128):
        raise ValueError(f"group {group} (32, 64 or 128)")
    if x.dim() < 1 or x.shape[-1] == 0 or x.shape[-1] % group:
        raise ValueError(f"x: the last dimension must be a positive multiple of the group of {group}")
    cols = x.shape[-1]
    if out is None:
        dtype = scale_dtype or (torch.bfloat16 if code == F32 else x.dtype)
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"scale_dtype: expected bfloat16 or float16, got {dtype}")
        scode = BF16 if dtype == torch.bfloat16 else F16
        lead, gs, u8 = x.shape[:-1], cols // group, torch.uint8
        out = INT4Tensor(_new_result((*lead, cols // 2), u8, dev, stream), _new_result((*lead, gs), dtype, dev, stream),
                         _new_result((*lead, gs), u8, dev, stream) if zeros else None, group)
    else:
        if out.group != group or out.codes.shape != (*x.shape[:-1], cols // 2) or (out.zeros is not None) != zeros or \
                (scale_dtype is not None and out.scales.dtype != scale_dtype):
            raise ValueError("out does not match x, group, zeros and scale_dtype")
        scode = _need_int4(out, "out", dev)
    if x.numel() == 0:
        return out
    _call(dev, stream, lib().int4_quantize, x.data_ptr(), code, x.numel() // cols, cols, group, scode,
          out.codes.data_ptr(), out.scales.data_ptr(), _ptr(out.zeros))
    return out


def int4_dequantize(q: INT4Tensor, out_dtype=None, out=None, stream=None):
    """The values of q [..., rows, cols] in its scales' type, or float32."""
    import torch
    dev = q.codes.device
    code = _need_int4(q, "q", dev)
    cols = 2 * q.codes.shape[-1]
    want = out.dtype if out is not None and out_dtype is None else (out_dtype or q.scales.dtype)
    if want not in (q.scales.dtype, torch.float32):
        raise TypeError(f"out: {q.scales.dtype} or float32, got {want}")
    out = _result(out, tuple(q.codes.shape[:-1]) + (cols,), want, q.codes, "out", stream)
    if out.numel() == 0:
        return out
    _call(dev, stream, lib().int4_dequantize, q.codes.data_ptr(), q.scales.data_ptr(), _ptr(q.zeros),
          out.numel() // cols, cols, q.group, code, F32 if want == torch.float32 else code, out.data_ptr())
    return out


def int4_grouped_gemv(a, b: INT4Tensor, offsets, *, m_total: int, a_rows=None, gated: bool = False,
                      activation: int = ACT_SILU, out=None, out_dtype=None, max_rows_per_expert_hint: int = 0,
                      stream=None):
    """Products of few rows with INT4 weights (see include/nvfp4moe.h): a bf16/f16
    [rows, K], b [E, N, K] with scales in a's type, offsets int32 [E+1] -> y
    [m_total, N] in a's type or float32; gated (N = 2I, gate rows first): h =
    act(gate) * up [m_total, I]."""
    import torch
    if a.dim() != 2 or b.codes.dim() != 3:
        raise ValueError("a must be [rows, K] and b [E, N, K]")
    dev = b.codes.device
    code = _need_int4(b, "b", dev)
    _need(a, b.scales.dtype, "a", dev)
    E = _group(b.codes, offsets, dev)
    N, K = b.codes.shape[1], 2 * b.codes.shape[2]
    if a.shape[1] != K or (gated and N % 2):
        raise ValueError("operand shapes disagree")
    _rows_of(a_rows, a, m_total, dev, "a")
    want = out.dtype if out is not None and out_dtype is None else (out_dtype or a.dtype)
    if want != a.dtype and (gated or want != torch.float32):
        raise TypeError(f"out: {a.dtype}{'' if gated else ' or float32'}, got {want}")
    out = _result(out, (m_total, N // 2 if gated else N), want, a, "out", stream)
    args = Int4GemvArgs(a=a.data_ptr(), dtype=code, a_rows=_ptr(a_rows), a_rows_total=a.shape[0],
                        b_codes=b.codes.data_ptr(), b_scales=b.scales.data_ptr(), b_zeros=_ptr(b.zeros), group=b.group,
                        offsets=offsets.data_ptr(), E=E, N=N, K=K, m_total=m_total, gated=int(gated),
                        activation=activation, out_dtype=F32 if want == torch.float32 else code,
                        max_rows_per_expert_hint=max_rows_per_expert_hint, out=out.data_ptr())
    _call(dev, stream, lib().int4_grouped_gemv, ctypes.byref(args))
    return out


# -------------------------------------------------------------------------- swiglu
def moe_swiglu(gate_up, g=None, out: NVFP4Tensor | None = None, workspace=None, stream=None) -> NVFP4Tensor:
    """gate_up float32/bf16 [M, 2I] -> NVFP4 h = silu(gate) * up."""
    import torch
    _need(gate_up, gate_up.dtype, "gate_up")
    M, N2 = gate_up.shape
    I = N2 // 2
    dev = gate_up.device
    if out is None:
        out = NVFP4Tensor(_new_result((M, I // 2), torch.uint8, dev, stream),
                          _new_result((M, I // 16), torch.uint8, dev, stream),
                          _new_result(1, torch.float32, dev, stream))
    if workspace is None:
        workspace = _new(lib().moe_swiglu_workspace_size(), torch.uint8, dev, stream)
    _check(lib().moe_swiglu(gate_up.data_ptr(), _dtype_code(gate_up), M, I, _ptr(g), _ptr(out.g),
                            out.codes.data_ptr(), out.scales.data_ptr(), workspace.data_ptr(), workspace.numel(),
                            _stream(stream)))
    return out


# ------------------------------------------------------------------------- combine
def moe_unpermute_combine(y, perm_of_assignment, topk_w, T: int, k: int, out=None, out_dtype=None, stream=None):
    """out[t] = sum_j topk_w[t, j] * y[perm_of_assignment[t*k + j]] (bf16 by default)."""
    import torch
    _need(y, y.dtype, "y")
    H = y.shape[1]
    if out is None:
        out = _result(None, (T, H), out_dtype or torch.bfloat16, y, "out", stream)
    if tuple(out.shape) != (T, H):
        raise ValueError(f"out: expected [{T}, {H}], got {list(out.shape)}")
    _need(out, out.dtype, "out")
    if perm_of_assignment is not None:
        _need(perm_of_assignment, torch.int32, "perm_of_assignment")
        if perm_of_assignment.numel() < T * k:
            raise ValueError(f"perm_of_assignment: {perm_of_assignment.numel()} values, expected T*k = {T * k}")
    elif y.shape[0] < T * k:
        raise ValueError(f"y has {y.shape[0]} rows, fewer than T*k = {T * k} (and no perm_of_assignment)")
    if topk_w is not None:
        _need(topk_w, torch.float32, "topk_w")
        if topk_w.numel() < T * k:
            raise ValueError(f"topk_w: {topk_w.numel()} values, expected T*k = {T * k}")
    _call(y.device, stream, lib().moe_unpermute_combine, y.data_ptr(), _dtype_code(y), _ptr(perm_of_assignment),
          _ptr(topk_w), T, k, H, out.data_ptr(), _dtype_code(out))
    return out


def moe_unpermute_combine_backward(dout, y, perm_of_assignment, topk_w, *, k: int | None = None, need_dy: bool = True,
                                   need_dw: bool = True, dy=None, d_topk_w=None, stream=None):
    """Gradients of moe_unpermute_combine from dout [T, H]: (dy [rows, H] in y's
    type, d_topk_w float32 [T, k]); None where not needed.  topk_w float32 [T, k], or
    None for a plain sum (weights of 1) of k rows a token; perm_of_assignment as in
    the forward call (None: row t*k + j), its entries in [0, rows) and all different.
    Rows of a new dy that no entry names are zero."""
    import torch
    if dout.dim() != 2 or y.dim() != 2 or (topk_w is not None and topk_w.dim() != 2):
        raise ValueError("dout must be [T, H], y [rows, H] and topk_w [T, k]")
    if k is None:
        if topk_w is None:
            raise ValueError("k is needed without topk_w")
        k = topk_w.shape[1]
    if not (need_dy or need_dw):
        raise ValueError("neither dy nor d_topk_w is needed")
    dev = y.device
    y_code, d_code = _dtype_code(y), _dtype_code(dout)
    _need(y, y.dtype, "y", dev)
    _need(dout, dout.dtype, "dout", dev)
    (T, H), rows = dout.shape, y.shape[0]
    if topk_w is not None:
        _need_shape(topk_w, (T, k), torch.float32, "topk_w", dev)
    if y.shape[1] != H:
        raise ValueError("operand shapes disagree")
    if perm_of_assignment is not None:
        _need_shape(perm_of_assignment, (T * k,), torch.int32, "perm_of_assignment", dev)
    elif rows < T * k:
        raise ValueError(f"y has {rows} rows, fewer than T*k = {T * k} (and no perm_of_assignment)")
    if need_dy:
        fresh = dy is None
        dy = _result(dy, (rows, H), y.dtype, y, "dy", stream)
        if fresh and rows > T * k:
            with torch.cuda.stream(stream):
                dy.zero_()
    else:
        dy = None
    d_topk_w = _result(d_topk_w, (T, k), torch.float32, y, "d_topk_w", stream) if need_dw else None
    _call(dev, stream, lib().moe_unpermute_combine_backward, dout.data_ptr(), d_code, y.data_ptr(), y_code, rows,
          _ptr(perm_of_assignment), _ptr(topk_w), T, k, H, _ptr(dy), _ptr(d_topk_w))
    return dy, d_topk_w


__all__ = ["lib", "moe_route_permute", "moe_route_quantize", "moe_route_quantize_noalloc", "nvfp4_quantize", "nvfp4_grouped_gemm", "moe_swiglu", "nvfp4_weight_repack",
           "moe_unpermute_combine", "moe_expert_ffn", "moe_expert_ffn_workspace", "mxfp4_quantize",
           "mxfp4_grouped_gemm", "mxfp4_weight_repack", "MXFP4Tensor", "fp8_quantize", "fp8_swiglu_quantize", "fp8_weight_repack",
           "fp8_grouped_gemm", "FP8Tensor", "Fp8GemmArgs", "NVFP4Tensor", "Routing", "GemmArgs", "NVFP4MoEError",
           "moe_gated_ffn", "moe_gated_ffn_backward", "moe_grouped_gemm", "moe_grouped_gemm_backward", "int8_quantize",
           "int8_grouped_gemm", "INT8Tensor", "moe_route_scored", "moe_route_scored_backward",
           "moe_unpermute_combine_backward", "int4_quantize", "int4_dequantize", "int4_grouped_gemv", "INT4Tensor",
           "SCORE_SOFTMAX", "SCORE_SIGMOID", "ACT_SILU", "ACT_GELU", "F16", "EPI_SWIGLU_BF16",
           "F32", "BF16", "EPI_F32", "EPI_BF16", "EPI_SWIGLU_NVFP4", "EPI_COMBINE_F32"]

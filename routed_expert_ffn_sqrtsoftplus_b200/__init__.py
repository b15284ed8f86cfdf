"""B200 (sm_100a) DeepSeek-V4.1-Flash routed-expert FFN layer with sqrtsoftplus routing.

A thin ctypes binding of the C ABI in include/moe.h. It only marshals torch
tensors into pointers and streams: every step of the layer runs in the CUDA
kernels of libmoe_b200.so. There is no CPU fallback; if the library is missing
or no CUDA device is present the calls raise.

    from routed_expert_ffn_sqrtsoftplus_b200 import MoELayer
    layer = MoELayer(hidden=5120, inter=2304, n_routed=384, n_shared=1, top_k=6,
                     max_tokens=32, router_w=wg, w1=w1, w3=w3, w2=w2,
                     sh_w1=s1, sh_w3=s3, sh_w2=s2)
    y = layer(x)                       # x, y: BF16 [T, 5120] on the GPU
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmoe_b200.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_OOM, MOE_ERR_CUDA, MOE_ERR_TIMEOUT, MOE_ERR_DEVICE = range(7)
MOE_DT_BF16, MOE_DT_MXFP4, MOE_DT_MXFP8 = 0, 1, 2

# moe_buffer ids
(BUF_LOGITS, BUF_TOPK_IDX, BUF_TOPK_W, BUF_COUNTS, BUF_OFFSETS, BUF_PERM, BUF_INV, BUF_H, BUF_XQ, BUF_XQ_SCALES,
 BUF_HQ, BUF_HQ_SCALES, BUF_NTILES, BUF_TILES_GU, BUF_TILES_DN) = range(15)

EXPORTED = ("moe_create", "moe_forward", "moe_forward_host", "moe_get_status", "moe_status_string",
            "moe_destroy", "moe_abi_version", "moe_quantize_mxfp4", "moe_inspect", "moe_set_wait_timeout",
            "moe_selftest_wait_timeout", "moe_get_info", "moe_profile_begin", "moe_profile_end",
            "moe_num_kernel_kinds", "moe_kernel_name", "moe_route_noalloc", "moe_quantize_mxfp8",
            "moe_set_hash_table", "moe_forward_hashed", "moe_fill_workspace", "moe_create_ep",
            "moe_forward_partial", "moe_read_bandwidth", "moe_forward_host_async", "moe_forward_host_wait",
            "moe_route", "moe_route_backward", "moe_forward_routed", "moe_quantize_fp4", "moe_dequantize_fp4",
            "moe_fp4_pad_scales", "moe_fp4_workspace_bytes", "moe_fp4_matmul",
            "moe_fp4_linear_workspace_bytes", "moe_fp4_linear", "moe_fp4_set_wait_timeout",
            "moe_fp4_get_status")

SCORES = {"softmax": 0, "sigmoid": 1, "sqrtsoftplus": 2}
FP4_FORMATS = {"mxfp4": 0, "nvfp4": 1}
FP4_BLOCK = {"mxfp4": 32, "nvfp4": 16}   # values of K per scale
_VALUE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        name = _status_name(status)
        super().__init__(f"{what}: {name}" if what else name)


class _Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_routed", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("top_k", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("route_scale", ctypes.c_float), ("swiglu_limit", ctypes.c_float),
                ("expert_dtype", ctypes.c_int32)]


class _Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("router_w", "router_bias", "w1", "w3", "w2", "s1", "s3", "s2",
                                              "sh_w1", "sh_w3", "sh_w2")]


class _Info(ctypes.Structure):
    _fields_ = [("weight_bytes", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64),
                ("num_sms", ctypes.c_int32), ("last_tokens", ctypes.c_int32)]


class _RouteConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_experts", "top_k", "n_groups", "topk_groups", "score", "group_top2",
                                             "renormalize")] + [("route_scale", ctypes.c_float)]


class _Fp4Product(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("format", "T", "N", "K", "E", "out_dtype")] +
                [("x", ctypes.c_void_p), ("x_scales", ctypes.c_void_p), ("x_scale_stride", ctypes.c_int64),
                 ("x_tensor_scale", ctypes.c_void_p), ("w", ctypes.c_void_p), ("w_scales", ctypes.c_void_p),
                 ("w_scale_stride", ctypes.c_int64)] +
                [(n, ctypes.c_void_p) for n in ("w_tensor_scale", "offsets", "y", "workspace")] +
                [("workspace_bytes", ctypes.c_int64), ("status", ctypes.c_void_p)])


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmoe_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m routed_expert_ffn_sqrtsoftplus_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, U64, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_int64
        sig = {
            "moe_create": (I32, [ctypes.POINTER(_Config), ctypes.POINTER(_Weights), P, ctypes.POINTER(P)]),
            "moe_forward": (I32, [P, P, I32, P, P, P, P]),
            "moe_forward_host": (I32, [P, P, I32, P, P, P, P]),
            "moe_forward_host_async": (I32, [P, P, I32, P, P]),
            "moe_forward_host_wait": (I32, [P, P]),
            "moe_get_status": (I32, [P]),
            "moe_status_string": (ctypes.c_char_p, [I32]),
            "moe_destroy": (None, [P]),
            "moe_abi_version": (I32, []),
            "moe_quantize_mxfp4": (I32, [P, I64, I32, P, P, P]),
            "moe_quantize_mxfp8": (I32, [P, I64, I32, P, P, P]),
            "moe_set_hash_table": (I32, [P, P, I32, P]),
            "moe_fill_workspace": (I32, [P, I32, P]),
            "moe_create_ep": (I32, [ctypes.POINTER(_Config), ctypes.POINTER(_Weights), I32, I32, P,
                                    ctypes.POINTER(P)]),
            "moe_forward_partial": (I32, [P, P, I32, P, P, P, P]),
            "moe_read_bandwidth": (I32, [P, ctypes.c_size_t, I32, P, ctypes.POINTER(ctypes.c_double)]),
            "moe_forward_hashed": (I32, [P, P, P, I32, P, P, P, P]),
            "moe_inspect": (I32, [P, I32, P, ctypes.c_size_t, P]),
            "moe_set_wait_timeout": (I32, [P, U64]),
            "moe_selftest_wait_timeout": (I32, [P, U64, P]),
            "moe_get_info": (I32, [P, ctypes.POINTER(_Info)]),
            "moe_profile_begin": (I32, [P, I32]),
            "moe_profile_end": (I32, [P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(I64), I32]),
            "moe_num_kernel_kinds": (I32, []),
            "moe_kernel_name": (ctypes.c_char_p, [I32]),
            "moe_route_noalloc": (I32, [P, P, P, I32, I32, I32, I32, ctypes.c_float, P, P, P]),
            "moe_route": (I32, [ctypes.POINTER(_RouteConfig), P, I32, I64, P, I32, P, P, P]),
            "moe_route_backward": (I32, [ctypes.POINTER(_RouteConfig), P, P, I32, I64, P, I32, P, P]),
            "moe_forward_routed": (I32, [P, P, P, P, I32, P, P]),
            "moe_quantize_fp4": (I32, [I32, P, I32, I64, I32, I64, P, P, P, I64, P]),
            "moe_dequantize_fp4": (I32, [I32, P, P, I64, I32, I64, P, P, I32, P]),
            "moe_fp4_pad_scales": (I32, [P, I64, I32, P, I64, P]),
            "moe_fp4_workspace_bytes": (I64, [I32, I32, I32, I32, I32]),
            "moe_fp4_matmul": (I32, [ctypes.POINTER(_Fp4Product), P]),
            "moe_fp4_linear_workspace_bytes": (I64, [I32, I32, I32, I32, I32]),
            "moe_fp4_linear": (I32, [ctypes.POINTER(_Fp4Product), I32, I64, P]),
            "moe_fp4_set_wait_timeout": (I32, [U64]),
            "moe_fp4_get_status": (I32, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _status_name(s: int) -> str:
    try:
        return lib().moe_status_string(s).decode()
    except Exception:
        return f"status {s}"


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoEError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _need(t: torch.Tensor, name: str, dtype, shape=None, device_type="cuda"):
    if t.device.type != device_type:
        raise ValueError(f"{name} must be on {device_type}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def kernel_names():
    L = lib()
    return [L.moe_kernel_name(i).decode() for i in range(L.moe_num_kernel_kinds())]


def quantize_mxfp4(w: torch.Tensor, stream=None):
    """BF16 [..., K] (CUDA) -> (packed E2M1 uint8 [..., K/2], E8M0 uint8 [..., K/32]) on the device."""
    _need(w, "w", torch.bfloat16)
    K = w.shape[-1]
    rows = w.numel() // K
    packed = torch.empty(w.shape[:-1] + (K // 2,), dtype=torch.uint8, device=w.device)
    scales = torch.empty(w.shape[:-1] + (K // 32,), dtype=torch.uint8, device=w.device)
    _check(lib().moe_quantize_mxfp4(_ptr(w), rows, K, _ptr(packed), _ptr(scales), _stream(stream)),
           "moe_quantize_mxfp4")
    return packed, scales


def quantize_mxfp8(w: torch.Tensor, stream=None):
    """BF16 [..., K] (CUDA) -> (E4M3 codes uint8 [..., K], E8M0 uint8 [..., K/32]) on the device."""
    _need(w, "w", torch.bfloat16)
    K = w.shape[-1]
    rows = w.numel() // K
    codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    scales = torch.empty(w.shape[:-1] + (K // 32,), dtype=torch.uint8, device=w.device)
    _check(lib().moe_quantize_mxfp8(_ptr(w), rows, K, _ptr(codes), _ptr(scales), _stream(stream)),
           "moe_quantize_mxfp8")
    return codes, scales


def read_bandwidth(buf: torch.Tensor, reps: int = 5, stream=None) -> float:
    """Read-only streaming bandwidth (GB/s) of the device holding `buf` (a large CUDA tensor)."""
    if buf.device.type != "cuda" or not buf.is_contiguous():
        raise ValueError("buf must be a contiguous CUDA tensor")
    g = ctypes.c_double(0.0)
    _check(lib().moe_read_bandwidth(_ptr(buf), buf.numel() * buf.element_size(), reps, _stream(stream),
                                    ctypes.byref(g)), "moe_read_bandwidth")
    return g.value


# ------------------------------------------------------------------ operators without a handle
# With `stream`, the whole call runs on it (its outputs and workspaces belong to it as well).
def _on_stream(stream):
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream)))


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _current(t: torch.Tensor) -> int:
    return torch._C._cuda_getCurrentRawStream(t.device.index)


# A call's time on few rows is the host's: an output through new_empty takes 1.9 us of it, through the
# allocator's own entry 0.8 (on the current device, where the library wants every tensor to be). That entry passes by
# the dispatcher: not under a dispatch mode, for tensors of other classes, or where fresh memory is to be filled.
try:
    from torch._C import _cuda_getDevice, _get_deterministic_algorithms, _len_torch_dispatch_stack
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None
_PLAIN = (torch.Tensor, torch.nn.Parameter)


def _empty(ref: torch.Tensor, rows: int, cols: int, dtype) -> torch.Tensor:
    """A matrix for a call's results, on ref's device."""
    if (_empty_strided_cuda is None or type(ref) not in _PLAIN or ref.get_device() != _cuda_getDevice() or
            _len_torch_dispatch_stack() or _get_deterministic_algorithms()):
        return ref.new_empty((rows, cols), dtype=dtype)
    return _empty_strided_cuda((rows, cols), (cols, 1), dtype)


def _bytes(ref: torch.Tensor, n: int) -> torch.Tensor:
    """A workspace of n bytes."""
    return _empty(ref, 1, n, torch.uint8)


def _arg(t: torch.Tensor, name: str, dtype, shape, ref: torch.Tensor):
    """A contiguous tensor of this type and shape (None: any), on ref's device."""
    if t.dtype != dtype or t.get_device() != ref.get_device() or not t.is_contiguous() or (
            shape is not None and t.shape != shape):
        _need(t, name, dtype, shape, ref.device.type)
        raise ValueError(f"{name} is on {t.device}, expected {ref.device}")


def _rows(t: torch.Tensor, name: str):
    """A CUDA matrix of a supported value type with contiguous rows: (rows, cols, row stride, dtype code)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be on cuda")
    code = _VALUE_DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got {t.dim()}")
    (r, c), (rs, cs) = t.shape, t.stride()
    if r >= 1 << 31 or c >= 1 << 31:
        raise ValueError(f"{name} must have fewer than 2^31 rows and columns")
    if c > 1 and cs != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if r <= 1:
        rs = c
    elif rs < c:
        raise ValueError(f"{name} must not have overlapping rows")
    return r, c, rs, code


@functools.lru_cache(maxsize=1024)
def _route_config(E, k, n_groups, topk_groups, score, group_score, renormalize, route_scale):
    if score not in SCORES:
        raise ValueError(f"score must be one of {tuple(SCORES)}")
    if group_score not in ("top2", "max"):
        raise ValueError("group_score must be 'top2' or 'max'")
    if not 1 <= k <= E or max(abs(n_groups), abs(topk_groups)) >= 1 << 31:
        raise ValueError(f"top_k must be 1 .. {E}, got {k}, with fewer than 2^31 groups")
    return _RouteConfig(E, k, n_groups, topk_groups, SCORES[score], group_score == "top2", bool(renormalize),
                        route_scale)


def route(logits: torch.Tensor, top_k: int, *, score: str = "softmax", bias: Optional[torch.Tensor] = None,
          n_groups: int = 1, topk_groups: int = 1, group_score: str = "top2", renormalize: bool = True,
          route_scale: float = 1.0, topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
          stream=None):
    """Routing from logits [T, E] (bfloat16, float16 or float32): (topk_idx int32 [T, k], topk_w fp32 [T, k]).

    The k experts with the largest score + bias, from the topk_groups worthiest of n_groups groups of
    consecutive experts (worth: the largest key, or with group_score "top2" the sum of the two largest), in
    descending order, lower expert first on a tie; the weights are the scores without the bias, divided by their
    sum with ``renormalize``, times route_scale. A logit of -inf takes its expert out; a slot without an expert
    has index -1 and weight 0. A row that is not finite (NaN or +inf) gets experts 0..k-1 with NaN weights.

    Where autograd records and the logits require grad, the weights carry their graph (route_backward; the bias only
    selects and gets no gradient); topk_idx and topk_w may not be given then, as with torch's out arguments. As with
    torch's own operators, a step that is captured with its backward pass needs leaves of which no eager graph lives on.
    """
    if stream is not None:
        with _on_stream(stream):
            return route(logits, top_k, score=score, bias=bias, n_groups=n_groups, topk_groups=topk_groups,
                         group_score=group_score, renormalize=renormalize, route_scale=route_scale,
                         topk_idx=topk_idx, topk_w=topk_w)
    if logits.requires_grad and torch.is_grad_enabled():
        if topk_idx is not None or topk_w is not None:
            raise ValueError("topk_idx and topk_w may not be given where the logits require grad")
        return _Route.apply(logits, top_k, score, bias, n_groups, topk_groups, group_score, renormalize, route_scale)
    T, E, rs, code = _rows(logits, "logits")
    if bias is not None:
        _arg(bias, "bias", torch.float32, (E,), logits)
    cfg = _route_config(E, top_k, n_groups, topk_groups, score, group_score, renormalize, route_scale)
    if topk_idx is None:
        topk_idx = _empty(logits, T, top_k, torch.int32)
    else:
        _arg(topk_idx, "topk_idx", torch.int32, (T, top_k), logits)
    if topk_w is None:
        topk_w = _empty(logits, T, top_k, torch.float32)
    else:
        _arg(topk_w, "topk_w", torch.float32, (T, top_k), logits)
    _check(lib().moe_route(cfg, logits.data_ptr(), code, rs, _addr(bias), T, topk_idx.data_ptr(),
                           topk_w.data_ptr(), _current(logits)), "moe_route")
    return topk_idx, topk_w


def route_backward(grad_w: torch.Tensor, logits: torch.Tensor, topk_idx: torch.Tensor, *, score: str = "softmax",
                   renormalize: bool = True, route_scale: float = 1.0, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Gradient of the logits [T, E] (in their dtype) from that of route()'s weights, the selection held fixed."""
    if stream is not None:
        with _on_stream(stream):
            return route_backward(grad_w, logits, topk_idx, score=score, renormalize=renormalize,
                                  route_scale=route_scale, out=out)
    T, E, rs, code = _rows(logits, "logits")
    k = topk_idx.shape[-1]
    _arg(topk_idx, "topk_idx", torch.int32, (T, k), logits)
    _arg(grad_w, "grad_w", torch.float32, (T, k), logits)
    cfg = _route_config(E, k, 1, 1, score, "max", renormalize, route_scale)
    if out is None:
        out = _empty(logits, T, E, logits.dtype)
    else:
        _arg(out, "out", logits.dtype, (T, E), logits)
    _check(lib().moe_route_backward(cfg, grad_w.data_ptr(), logits.data_ptr(), code, rs, topk_idx.data_ptr(), T,
                                    out.data_ptr(), _current(logits)), "moe_route_backward")
    return out


class _Route(torch.autograd.Function):
    """route() in a graph: the selection is held fixed, the weights' gradient becomes the logits'."""

    @staticmethod
    def forward(ctx, logits, top_k, score, bias, n_groups, topk_groups, group_score, renormalize, route_scale):
        idx, w = route(logits, top_k, score=score, bias=bias, n_groups=n_groups, topk_groups=topk_groups,
                       group_score=group_score, renormalize=renormalize, route_scale=route_scale)
        ctx.mark_non_differentiable(idx)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(logits, idx)
        ctx.how = score, renormalize, route_scale
        return idx, w

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, grad_w):
        if grad_w is None:
            return (None,) * 9
        logits, idx = ctx.saved_tensors
        score, renormalize, route_scale = ctx.how
        return (route_backward(grad_w.contiguous(), logits, idx, score=score, renormalize=renormalize,
                               route_scale=route_scale),) + (None,) * 8


def _fp4_format(fmt: str) -> int:
    if fmt not in FP4_FORMATS:
        raise ValueError(f"fmt must be one of {tuple(FP4_FORMATS)}")
    return FP4_FORMATS[fmt]


def _tensor_scale(t: Optional[torch.Tensor], name: str, fmt: str, n: int, ref: torch.Tensor):
    if t is None:
        return None
    if fmt != "nvfp4":
        raise ValueError(f"{name} is for nvfp4")
    if t.numel() != n:
        raise ValueError(f"{name} must hold {n} value(s), got {t.numel()}")
    _arg(t, name, torch.float32, None, ref)
    return t.data_ptr()


def quantize_fp4(x: torch.Tensor, fmt: str, tensor_scale: Optional[torch.Tensor] = None, stream=None):
    """x [rows, K] (bfloat16, float16 or float32; K % 32 == 0) -> (codes uint8 [rows, K/2], scales uint8).

    fmt "mxfp4": scales E8M0 [rows, K/32], the rule of quantize_mxfp4. fmt "nvfp4": scales E4M3 [rows, K/16],
    relative to tensor_scale (fp32, one value; 1 when None). Element 2j is the low nibble of byte j.
    """
    if stream is not None:
        with _on_stream(stream):
            return quantize_fp4(x, fmt, tensor_scale)
    f = _fp4_format(fmt)
    rows, K, rs, code = _rows(x, "x")
    if K % 32 != 0:
        raise ValueError(f"x must have a multiple of 32 columns, got {K}")
    ts = _tensor_scale(tensor_scale, "tensor_scale", fmt, 1, x)
    sc = K // FP4_BLOCK[fmt]
    codes = _empty(x, rows, K // 2, torch.uint8)
    scales = _empty(x, rows, sc, torch.uint8)
    _check(lib().moe_quantize_fp4(f, x.data_ptr(), code, rows, K, rs, ts, codes.data_ptr(), scales.data_ptr(), sc,
                                  _current(x)), "moe_quantize_fp4")
    return codes, scales


def dequantize_fp4(codes: torch.Tensor, scales: torch.Tensor, fmt: str, tensor_scale: Optional[torch.Tensor] = None,
                   dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The values [rows, K] that codes [rows, K/2] and scales stand for, in fp32, rounded to dtype."""
    if stream is not None:
        with _on_stream(stream):
            return dequantize_fp4(codes, scales, fmt, tensor_scale, dtype)
    f = _fp4_format(fmt)
    if dtype not in _VALUE_DTYPES:
        raise ValueError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    if codes.dim() != 2:
        raise ValueError(f"codes must have 2 dimensions, got {codes.dim()}")
    rows, K = codes.shape[0], codes.shape[1] * 2
    _need(codes, "codes", torch.uint8)
    if K >= 1 << 31:
        raise ValueError("codes must have fewer than 2^30 columns")
    if K % 32 != 0:
        raise ValueError(f"codes must have a multiple of 16 columns, got {codes.shape[1]}")
    _arg(scales, "scales", torch.uint8, (rows, K // FP4_BLOCK[fmt]), codes)
    ts = _tensor_scale(tensor_scale, "tensor_scale", fmt, 1, codes)
    out = _empty(codes, rows, K, dtype)
    _check(lib().moe_dequantize_fp4(f, codes.data_ptr(), scales.data_ptr(), rows, K, scales.shape[1], ts,
                                    out.data_ptr(), _VALUE_DTYPES[dtype], _current(codes)), "moe_dequantize_fp4")
    return out


def _fp4_weights(w, w_scales, fmt, K, offsets, ref):
    """(E, N) of w [N, K/2] or, with offsets, [E, N, K/2]."""
    lead = w.shape[:-1]
    if w.dim() != (2 if offsets is None else 3) or w.shape[-1] * 2 != K:
        raise ValueError(f"w must be [{'' if offsets is None else 'E, '}N, {K // 2}], got {tuple(w.shape)}")
    _arg(w, "w", torch.uint8, None, ref)
    _arg(w_scales, "w_scales", torch.uint8, lead + (K // FP4_BLOCK[fmt],), ref)
    if offsets is None:
        return 1, lead[0]
    _arg(offsets, "offsets", torch.int32, (lead[0] + 1,), ref)
    return lead


def _fp4_out(x, T, N, out, out_dtype):
    if out is None:
        return _empty(x, T, N, out_dtype)
    if out.dtype not in _VALUE_DTYPES:
        raise ValueError(f"out must be bfloat16, float16 or float32, got {out.dtype}")
    _arg(out, "out", out.dtype, (T, N), x)
    return out


def _aligned_scales(scales, f):
    """(scales, row stride) with rows that a product without a workspace can read: as they are, or padded copies."""
    cols = scales.shape[-1]
    if (cols | scales.data_ptr()) % (16 if f else 8) == 0:
        return scales, cols
    rows, stride = scales.numel() // cols, (cols + 15) // 16 * 16
    padded = scales.new_empty((rows, stride))
    _check(lib().moe_fp4_pad_scales(scales.data_ptr(), rows, cols, padded.data_ptr(), stride, _current(scales)),
           "moe_fp4_pad_scales")
    return padded, stride


@functools.lru_cache(maxsize=4096)
def _fp4_workspace_bytes(linear, device, *shape):
    if max(shape) >= 1 << 31:
        raise ValueError("an FP4 product takes fewer than 2^31 rows, columns and experts")
    L = lib()
    return (L.moe_fp4_linear_workspace_bytes if linear else L.moe_fp4_workspace_bytes)(*shape)


def _workspace_size(linear, f, T, N, K, E):
    # kept by the device that the library plans for: the current one, which need not be the tensors' (a call that is refused)
    return _fp4_workspace_bytes(linear, torch._C._cuda_getDevice(), f, T, N, K, E)


def fp4_set_wait_timeout(ns: int):
    """Limit of the device-side waits of the FP4 products from now on (the process's; default 2 s)."""
    if not 1 <= ns < 1 << 64:
        raise ValueError(f"the limit must be 1 .. 2^64 - 1 ns, got {ns}")
    _check(lib().moe_fp4_set_wait_timeout(ns), "moe_fp4_set_wait_timeout")


def fp4_status() -> int:
    """Whether a device-side wait ran out in FP4 products on the current device that were given no status word
    (MOE_OK or MOE_ERR_TIMEOUT); synchronises the device, and clears it."""
    return lib().moe_fp4_get_status()


def fp4_matmul(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, fmt: str, *,
               x_tensor_scale: Optional[torch.Tensor] = None, w_tensor_scale: Optional[torch.Tensor] = None,
               offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               out_dtype: torch.dtype = torch.bfloat16, status: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """y [T, N] = x w^T over the values of FP4 codes (quantize_fp4's): x [T, K/2], w [N, K/2].

    With offsets (int32 [E + 1], on the device) w is [E, N, K/2] and rows offsets[g] .. offsets[g + 1] of x meet
    w[g]; rows in no range are left as they were in ``out`` (not set where out is None). w_tensor_scale: one value
    per expert. status: int32 [1], set to 1 if a device-side wait ran out (without it fp4_status() tells); elements of
    y are then right or left as they were.
    """
    if stream is not None:
        with _on_stream(stream):
            return fp4_matmul(x, x_scales, w, w_scales, fmt, x_tensor_scale=x_tensor_scale,
                              w_tensor_scale=w_tensor_scale, offsets=offsets, out=out, out_dtype=out_dtype,
                              status=status)
    f = _fp4_format(fmt)
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dimensions, got {x.dim()}")
    if out is None and out_dtype not in _VALUE_DTYPES:
        raise ValueError(f"out_dtype must be bfloat16, float16 or float32, got {out_dtype}")
    T, K = x.shape[0], x.shape[1] * 2
    _need(x, "x", torch.uint8)
    if K % 32 != 0:
        raise ValueError(f"x must have a multiple of 16 columns, got {x.shape[1]}")
    _arg(x_scales, "x_scales", torch.uint8, (T, K // FP4_BLOCK[fmt]), x)
    E, N = _fp4_weights(w, w_scales, fmt, K, offsets, x)
    x_ts = _tensor_scale(x_tensor_scale, "x_tensor_scale", fmt, 1, x)
    w_ts = _tensor_scale(w_tensor_scale, "w_tensor_scale", fmt, E, x)
    out = _fp4_out(x, T, N, out, out_dtype)
    if status is not None:
        _arg(status, "status", torch.int32, (1,), x)
    xss, wss = x_scales.shape[1], w_scales.shape[-1]
    nbytes = _workspace_size(False, f, T, N, K, E)
    if nbytes == 0:       # the scales are read as they are: aligned rows
        w_scales, wss = _aligned_scales(w_scales, f)
        x_scales, xss = _aligned_scales(x_scales, f)
    space = _bytes(x, nbytes) if nbytes else None
    p = _Fp4Product(f, T, N, K, E, _VALUE_DTYPES[out.dtype], x.data_ptr(), x_scales.data_ptr(), xss, x_ts,
                    w.data_ptr(), w_scales.data_ptr(), wss, w_ts, _addr(offsets), out.data_ptr(), _addr(space), nbytes,
                    _addr(status))
    _check(lib().moe_fp4_matmul(p, _current(x)), "moe_fp4_matmul")
    return out


def fp4_linear(x: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, fmt: str, *,
               x_tensor_scale: Optional[torch.Tensor] = None, w_tensor_scale: Optional[torch.Tensor] = None,
               offsets: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = x w^T with x [T, K] (bfloat16, float16 or float32) quantised to fmt first, then fp4_matmul.

    w, w_scales, the tensor scales, offsets, out and status as there; y has x's dtype unless out says otherwise, and
    no graph.
    """
    if stream is not None:
        with _on_stream(stream):
            return fp4_linear(x, w, w_scales, fmt, x_tensor_scale=x_tensor_scale, w_tensor_scale=w_tensor_scale,
                              offsets=offsets, out=out, status=status)
    f = _fp4_format(fmt)
    T, K, rs, code = _rows(x, "x")
    if K % 32 != 0:
        raise ValueError(f"x must have a multiple of 32 columns, got {K}")
    E, N = _fp4_weights(w, w_scales, fmt, K, offsets, x)
    x_ts = _tensor_scale(x_tensor_scale, "x_tensor_scale", fmt, 1, x)
    w_ts = _tensor_scale(w_tensor_scale, "w_tensor_scale", fmt, E, x)
    out = _fp4_out(x, T, N, out, x.dtype)
    if status is not None:
        _arg(status, "status", torch.int32, (1,), x)
    wss = w_scales.shape[-1]
    # scales that are read as they are; rows that no base aligns the call itself copies
    if w_scales.data_ptr() % 16 != 0 and wss % (16 if f else 8) == 0 and (
            _workspace_size(False, f, T, N, K, E) == 0):
        w_scales, wss = _aligned_scales(w_scales, f)
    nbytes = _workspace_size(True, f, T, N, K, E)
    space = _bytes(x, nbytes)
    p = _Fp4Product(f, T, N, K, E, _VALUE_DTYPES[out.dtype], x.data_ptr(), None, 0, x_ts, w.data_ptr(),
                    w_scales.data_ptr(), wss, w_ts, _addr(offsets), out.data_ptr(), space.data_ptr(), nbytes,
                    _addr(status))
    _check(lib().moe_fp4_linear(p, code, rs, _current(x)), "moe_fp4_linear")
    return out


class MoELayer:
    """One routed-expert FFN layer resident on the current CUDA device."""

    def __init__(self, *, hidden: int, inter: int, n_routed: int, n_shared: int, top_k: int, max_tokens: int,
                 router_w: torch.Tensor, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor,
                 sh_w1: Optional[torch.Tensor] = None, sh_w3: Optional[torch.Tensor] = None,
                 sh_w2: Optional[torch.Tensor] = None, router_bias: Optional[torch.Tensor] = None,
                 s1: Optional[torch.Tensor] = None, s3: Optional[torch.Tensor] = None,
                 s2: Optional[torch.Tensor] = None, route_scale: float = 1.5, swiglu_limit: float = 10.0,
                 expert_dtype: str = "bf16", expert_begin: int = 0, expert_count: Optional[int] = None,
                 stream=None):
        """expert_begin / expert_count: hold only that window of the routed experts
        (expert parallelism; w1 / w3 / w2 and s1 / s3 / s2 then hold expert_count
        experts); such a layer computes partial outputs only (forward_partial)."""
        self._h = ctypes.c_void_p(None)
        L = lib()
        H, I, E, S = hidden, inter, n_routed, n_shared
        Ec = E if expert_count is None else expert_count
        _need(router_w, "router_w", torch.bfloat16, (E, H))
        if router_bias is not None:
            _need(router_bias, "router_bias", torch.float32, (E,))
        if expert_dtype == "bf16":
            _need(w1, "w1", torch.bfloat16, (Ec, I, H)); _need(w3, "w3", torch.bfloat16, (Ec, I, H))
            _need(w2, "w2", torch.bfloat16, (Ec, H, I))
            dt = MOE_DT_BF16
        elif expert_dtype in ("mxfp4", "mxfp8"):
            div = 2 if expert_dtype == "mxfp4" else 1
            _need(w1, "w1", torch.uint8, (Ec, I, H // div)); _need(w3, "w3", torch.uint8, (Ec, I, H // div))
            _need(w2, "w2", torch.uint8, (Ec, H, I // div))
            for n, t, shp in (("s1", s1, (Ec, I, H // 32)), ("s3", s3, (Ec, I, H // 32)),
                              ("s2", s2, (Ec, H, I // 32))):
                if t is None:
                    raise ValueError(f"{n} is required for {expert_dtype} experts")
                _need(t, n, torch.uint8, shp)
            dt = MOE_DT_MXFP4 if expert_dtype == "mxfp4" else MOE_DT_MXFP8
        else:
            raise ValueError("expert_dtype must be 'bf16', 'mxfp4' or 'mxfp8'")
        if S > 0:
            _need(sh_w1, "sh_w1", torch.bfloat16, (S, I, H)); _need(sh_w3, "sh_w3", torch.bfloat16, (S, I, H))
            _need(sh_w2, "sh_w2", torch.bfloat16, (S, H, I))
        self.cfg = _Config(H, I, E, S, top_k, max_tokens, float(route_scale), float(swiglu_limit), dt)
        wts = _Weights(_ptr(router_w), _ptr(router_bias), _ptr(w1), _ptr(w3), _ptr(w2), _ptr(s1), _ptr(s3),
                       _ptr(s2), _ptr(sh_w1), _ptr(sh_w3), _ptr(sh_w2))
        st = _stream(stream)
        if expert_count is None and expert_begin == 0:
            _check(L.moe_create(ctypes.byref(self.cfg), ctypes.byref(wts), st, ctypes.byref(self._h)), "moe_create")
        else:
            _check(L.moe_create_ep(ctypes.byref(self.cfg), ctypes.byref(wts), expert_begin, Ec, st,
                                   ctypes.byref(self._h)), "moe_create_ep")
        self.expert_begin, self.expert_count = expert_begin, Ec
        # The library copied the weights on `st`; wait so the caller may free its tensors.
        torch.cuda.synchronize()
        self.hidden, self.inter, self.n_routed, self.n_shared, self.top_k = H, I, E, S, top_k
        self.max_tokens = max_tokens
        self.device = router_w.device

    # ------------------------------------------------------------------ forward
    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, topk_idx: Optional[torch.Tensor] = None,
                topk_w: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        T = x.shape[0]
        _need(x, "x", torch.bfloat16, (T, self.hidden))
        if x.device != self.device:
            raise ValueError(f"x is on {x.device}, the layer on {self.device}")
        if out is None:
            out = torch.empty_like(x)
        _need(out, "out", torch.bfloat16, (T, self.hidden))
        if out.device != self.device:
            raise ValueError(f"out is on {out.device}, the layer on {self.device}")
        if topk_idx is not None:
            _need(topk_idx, "topk_idx", torch.int32, (T, self.top_k))
        if topk_w is not None:
            _need(topk_w, "topk_w", torch.float32, (T, self.top_k))
        _check(lib().moe_forward(self._h, _ptr(x), T, _ptr(out), _ptr(topk_idx), _ptr(topk_w), _stream(stream)),
               "moe_forward")
        return out

    __call__ = forward

    def forward_partial(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """This layer's share of an expert-parallel layer, fp32 [T, H]: the selected
        slots whose expert lies in its window (plus the shared experts it holds)."""
        T = x.shape[0]
        _need(x, "x", torch.bfloat16, (T, self.hidden))
        if out is None:
            out = torch.empty((T, self.hidden), dtype=torch.float32, device=x.device)
        _need(out, "out", torch.float32, (T, self.hidden))
        for n, t in (("x", x), ("out", out)):
            if t.device != self.device:
                raise ValueError(f"{n} is on {t.device}, the layer on {self.device}")
        _check(lib().moe_forward_partial(self._h, _ptr(x), T, _ptr(out), None, None, _stream(stream)),
               "moe_forward_partial")
        return out

    def set_hash_table(self, table: torch.Tensor, stream=None):
        """Vocabulary table int32 [vocab, top_k] of a hash-routed layer (copied by the library)."""
        _need(table, "table", torch.int32)
        if table.dim() != 2 or table.shape[1] != self.top_k:
            raise ValueError(f"table must be [vocab, {self.top_k}]")
        _check(lib().moe_set_hash_table(self._h, _ptr(table), table.shape[0], _stream(stream)),
               "moe_set_hash_table")

    def forward_hashed(self, x: torch.Tensor, token_ids: torch.Tensor, out: Optional[torch.Tensor] = None,
                       topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
        """The layer with hash routing: experts from the table row of each token's id."""
        T = x.shape[0]
        _need(x, "x", torch.bfloat16, (T, self.hidden))
        _need(token_ids, "token_ids", torch.int32, (T,))
        if out is None:
            out = torch.empty_like(x)
        _need(out, "out", torch.bfloat16, (T, self.hidden))
        for n, t in (("x", x), ("token_ids", token_ids), ("out", out)):
            if t.device != self.device:
                raise ValueError(f"{n} is on {t.device}, the layer on {self.device}")
        if topk_idx is not None:
            _need(topk_idx, "topk_idx", torch.int32, (T, self.top_k))
        if topk_w is not None:
            _need(topk_w, "topk_w", torch.float32, (T, self.top_k))
        _check(lib().moe_forward_hashed(self._h, _ptr(x), _ptr(token_ids), T, _ptr(out), _ptr(topk_idx),
                                        _ptr(topk_w), _stream(stream)), "moe_forward_hashed")
        return out

    def forward_routed(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The layer with a given routing (route()'s, or any other): experts topk_idx int32 [T, top_k], -1 for an
        empty slot, with weights topk_w fp32 [T, top_k] as they are. As in every call of the layer y has no graph."""
        if stream is not None:
            with _on_stream(stream):
                return self.forward_routed(x, topk_idx, topk_w, out)
        T = x.shape[0]
        _need(x, "x", torch.bfloat16, (T, self.hidden))
        _need(topk_idx, "topk_idx", torch.int32, (T, self.top_k))
        _need(topk_w, "topk_w", torch.float32, (T, self.top_k))
        if out is None:
            out = torch.empty_like(x)
        _need(out, "out", torch.bfloat16, (T, self.hidden))
        for n, t in (("x", x), ("topk_idx", topk_idx), ("topk_w", topk_w), ("out", out)):
            if t.device != self.device:
                raise ValueError(f"{n} is on {t.device}, the layer on {self.device}")
        _check(lib().moe_forward_routed(self._h, _ptr(x), _ptr(topk_idx), _ptr(topk_w), T, _ptr(out),
                                        _stream(None)), "moe_forward_routed")
        return out

    def forward_with_routing(self, x: torch.Tensor, stream=None):
        T = x.shape[0]
        idx = torch.empty((T, self.top_k), dtype=torch.int32, device=x.device)
        w = torch.empty((T, self.top_k), dtype=torch.float32, device=x.device)
        y = self.forward(x, topk_idx=idx, topk_w=w, stream=stream)
        return y, idx, w

    def forward_host(self, x_host: torch.Tensor, y_host: torch.Tensor, topk_idx_host: Optional[torch.Tensor] = None,
                     topk_w_host: Optional[torch.Tensor] = None, stream=None):
        """Host buffers in, host buffers out (copies enqueued on the stream; sync before reading)."""
        T = x_host.shape[0]
        _need(x_host, "x_host", torch.bfloat16, (T, self.hidden), "cpu")
        _need(y_host, "y_host", torch.bfloat16, (T, self.hidden), "cpu")
        if topk_idx_host is not None:
            _need(topk_idx_host, "topk_idx_host", torch.int32, (T, self.top_k), "cpu")
        if topk_w_host is not None:
            _need(topk_w_host, "topk_w_host", torch.float32, (T, self.top_k), "cpu")
        _check(lib().moe_forward_host(self._h, _ptr(x_host), T, _ptr(y_host), _ptr(topk_idx_host),
                                      _ptr(topk_w_host), _stream(stream)), "moe_forward_host")

    def forward_host_async(self, x_host: torch.Tensor, y_host: torch.Tensor, stream=None):
        """Pipelined host buffers in and out: the copies run on the library's own streams
        and overlap the neighbouring calls' layers. Call forward_host_wait(stream) and
        synchronise the stream before reading y_host or reusing a call's buffers."""
        T = x_host.shape[0]
        _need(x_host, "x_host", torch.bfloat16, (T, self.hidden), "cpu")
        _need(y_host, "y_host", torch.bfloat16, (T, self.hidden), "cpu")
        _check(lib().moe_forward_host_async(self._h, _ptr(x_host), T, _ptr(y_host), _stream(stream)),
               "moe_forward_host_async")

    def forward_host_wait(self, stream=None):
        """Make the stream wait for every copy-out of forward_host_async so far."""
        _check(lib().moe_forward_host_wait(self._h, _stream(stream)), "moe_forward_host_wait")

    # ------------------------------------------------------------------ inspection
    def inspect(self, what: int, out: torch.Tensor, stream=None) -> torch.Tensor:
        nbytes = out.numel() * out.element_size()
        _check(lib().moe_inspect(self._h, what, _ptr(out), nbytes, _stream(stream)), "moe_inspect")
        return out

    def fill_workspace(self, byte_value: int, stream=None):
        """Overwrite every per-forward scratch buffer with one byte value (a debugging aid)."""
        _check(lib().moe_fill_workspace(self._h, int(byte_value), _stream(stream)), "moe_fill_workspace")

    def status(self) -> int:
        return lib().moe_get_status(self._h)

    def info(self) -> dict:
        i = _Info()
        _check(lib().moe_get_info(self._h, ctypes.byref(i)), "moe_get_info")
        return dict(weight_bytes=i.weight_bytes, workspace_bytes=i.workspace_bytes, num_sms=i.num_sms,
                    last_tokens=i.last_tokens)

    def set_wait_timeout(self, ns: int):
        _check(lib().moe_set_wait_timeout(self._h, int(ns)), "moe_set_wait_timeout")

    def selftest_wait_timeout(self, ns: int, stream=None):
        _check(lib().moe_selftest_wait_timeout(self._h, int(ns), _stream(stream)), "moe_selftest_wait_timeout")

    def profile_begin(self, max_calls: int):
        _check(lib().moe_profile_begin(self._h, max_calls), "moe_profile_begin")

    def profile_end(self) -> dict:
        L = lib()
        n = L.moe_num_kernel_kinds()
        ms = (ctypes.c_double * n)()
        cnt = (ctypes.c_int64 * n)()
        _check(L.moe_profile_end(self._h, ms, cnt, n), "moe_profile_end")
        return {kernel_names()[i]: (ms[i], cnt[i]) for i in range(n) if cnt[i] > 0}

    def close(self):
        if self._h:
            lib().moe_destroy(self._h)
            self._h = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @classmethod
    def from_layer(cls, layer: dict, *, top_k: int, max_tokens: int, route_scale: float = 1.5,
                   swiglu_limit: float = 10.0, mx: Optional[dict] = None, expert_window=None,
                   with_shared: bool = True, stream=None) -> "MoELayer":
        """Build from a dict of tensors (x ignored): wg, bias, w1, w3, w2, sh_w1, sh_w3, sh_w2.

        With ``mx`` = dict(w1, s1, w3, s3, w2, s2) of MXFP4 (packed, w1 [E, I, H/2]) or
        MXFP8 (w1 [E, I, H]) tensors the routed experts are stored in that format.
        """
        E, I, H = layer["w1"].shape
        S = layer["sh_w1"].shape[0] if (with_shared and layer.get("sh_w1") is not None) else 0
        sh = {n: (layer.get(n) if S > 0 else None) for n in ("sh_w1", "sh_w3", "sh_w2")}
        b, c = (0, None) if expert_window is None else expert_window
        if expert_window is not None and not (0 <= b and 1 <= c and b + c <= E):
            raise ValueError(f"expert window {expert_window} is not inside [0, {E})")
        cut = (lambda t: t) if expert_window is None else (lambda t: t[b:b + c].contiguous())
        kw = dict(hidden=H, inter=I, n_routed=E, n_shared=S, top_k=top_k, max_tokens=max_tokens,
                  router_w=layer["wg"], router_bias=layer.get("bias"), route_scale=route_scale,
                  swiglu_limit=swiglu_limit, expert_begin=b, expert_count=c, stream=stream, **sh)
        if mx is None:
            return cls(w1=cut(layer["w1"]), w3=cut(layer["w3"]), w2=cut(layer["w2"]), expert_dtype="bf16", **kw)
        fmt = "mxfp8" if mx["w1"].shape[-1] == H else "mxfp4"
        return cls(w1=cut(mx["w1"]), w3=cut(mx["w3"]), w2=cut(mx["w2"]), s1=cut(mx["s1"]), s3=cut(mx["s3"]),
                   s2=cut(mx["s2"]), expert_dtype=fmt, **kw)

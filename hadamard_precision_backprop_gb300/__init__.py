"""hadamard_precision_backprop_gb300: GB300 kernels of the HLQ/HOT backward pass.

The compute lives in ``libhlq.so`` (hand-written sm_103a CUDA behind the C
ABI of ``include/hlq.h``); this module is the thin Python binding: it
marshals torch tensors to pointers, allocates outputs and workspaces with
torch, and passes torch's current CUDA stream.  The operators around the layer
do the same in an extension module (``csrc/hlq_torch.cpp``) where a call's
arguments are all in order.  Every step of the path runs
in libhlq's kernels; there is no CPU or PyTorch fallback, and loading fails
loudly when the library has not been built.

Entry points (same names as the C ABI):
  hlq_compress_activation(x, rank)            -> (xbar int8 [Cin, T'], s_x)
  hlq_linear_backward_gx(g_y, w, ...)         -> g_x fp32 [T, Cin]
  hlq_linear_backward_gw(g_y, xbar, s_x, ...) -> g_w fp32 [Cout, Cin]
  hlq_layer_norm(x, w, b, ...)                -> y, mean, rstd (, x + residual)
  hlq_layer_norm_backward(g_y, x, ...)        -> g_x, g_weight, g_bias
  hlq_token_logprobs(logits, targets)         -> logp, lse fp32 [T]
  hlq_policy_loss(logits, actions, ...)       -> stats, logp, gradient of logits
  hlq_clip_grad_norm(grads, max_norm, ...)    -> norm and coefficient, grads clipped
  hlq_attention(q, k, v, ...)                 -> out, lse
  hlq_attention_backward(g_out, q, k, v, ...) -> g_q, g_k, g_v (or g_qkv)
  hlq_dropout(x, p, seed, ...)                -> y (+ residual)
  hlq_debug_gx_parts / hlq_debug_gw_parts     -> intermediates for checks
  hlq_workspace_bytes, hlq_read_device_status, hlq_status_string
"""
from __future__ import annotations

import array
import ctypes
import importlib.util
import os
import threading
import warnings

PER_TENSOR, PER_TOKEN = 0, 1
RNE, SR = 0, 1
F32, BF16 = 0, 1
OP_COMPRESS_ACTIVATION, OP_BACKWARD_GX, OP_BACKWARD_GW, OP_BACKWARD = 0, 1, 2, 3
OP_SELECT_GRANULARITY, OP_ABLATION_GW_HQ, OP_ABLATION_GX_HLA = 4, 5, 6
OP_BACKWARD_FUSED, OP_LAYER_STEP = 7, 8
XBAR_INT8, XBAR_INT4, XBAR_PER_CHANNEL = 8, 4, 0x100   # format word of the stored activation
DEV_NONFINITE, DEV_TIMEOUT, DEV_BADCODE = 0x1, 0x2, 0x4

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libhlq.so")

EXPORTS = [
    "hlq_workspace_bytes", "hlq_compress_activation", "hlq_linear_backward_gx",
    "hlq_linear_backward_gw", "hlq_debug_gx_parts", "hlq_debug_gw_parts",
    "hlq_read_device_status", "hlq_status_string", "hlq_version",
    "hlq_debug_hq_transform", "hlq_debug_hla_transform",
    "hlq_trace_begin", "hlq_trace_end", "hlq_trace_get", "hlq_trace_free",
    "hlq_debug_reference_gemm", "hlq_debug_tc_gemm", "hlq_debug_tc_gemm_ws_bytes",
    "hlq_linear_backward_gx_noalloc", "hlq_noalloc_scratch_bytes",
    "hlq_linear_backward",
    "hlq_layer_step_host",
    "hlq_layer_step_host_workspace_bytes",
    "hlq_select_gy_granularity",
    "hlq_ablation_gw_hq",
    "hlq_ablation_gx_hla",
    "hlq_linear_backward_fused",
    "hlq_layer_step",
    "hlq_debug_gemm_plan",
    "hlq_debug_wait_timeout",
    "hlq_set_gw_operands", "hlq_get_gw_operands", "hlq_debug_serialize_branches",
    "hlq_layer_norm", "hlq_layer_norm_backward", "hlq_layer_norm_backward_workspace_bytes",
    "hlq_token_logprobs", "hlq_policy_loss", "hlq_policy_loss_workspace_bytes",
    "hlq_clip_grad_norm", "hlq_clip_grad_norm_workspace_bytes",
    "hlq_attention", "hlq_attention_backward", "hlq_attention_backward_workspace_bytes",
    "hlq_dropout",
]

_lock = threading.Lock()
_lib = None


class HLQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def build_library(force: bool = False) -> str:
    """Compile libhlq.so in-tree (nvcc, sm_103a)."""
    from .build import build as _build
    return _build(force=force)


def lib() -> ctypes.CDLL:
    """The loaded libhlq (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libhlq is not built ({LIB_PATH} missing); run "
                "`python -m hadamard_precision_backprop_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, i64, i32, u64, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                ctypes.c_uint64, ctypes.c_size_t)
        f32 = ctypes.c_float
        sig = {
            "hlq_workspace_bytes": (sz, [i32, i64, i64, i64, i32, i32]),
            "hlq_compress_activation": (i32, [P, i32, i64, i64, i32, i32, i32, P,
                                              P, P, sz, P]),
            "hlq_linear_backward_gx": (i32, [P, P, i32, i64, i64, i64, i32, i32,
                                             i32, i32, u64, P, P, sz, P]),
            "hlq_linear_backward_gw": (i32, [P, i32, P, P, i64, i64, i64, i32,
                                             i32, i32, P, P, sz, P]),
            "hlq_debug_gx_parts": (i32, [P, P, i32, i64, i64, i64, i32, i32,
                                         i32, i32, u64, P, P, sz, P, P, P, P,
                                         P, P, P, P]),
            "hlq_debug_gw_parts": (i32, [P, i32, P, P, i64, i64, i64, i32, i32,
                                         i32, P, P, sz, P, P, P, P]),
            "hlq_read_device_status": (i32, [P, i32, P]),
            "hlq_debug_hq_transform": (i32, [P, i32, i64, i64, i32, P, P]),
            "hlq_debug_hla_transform": (i32, [P, i32, i64, i64, i32, P, P]),
            "hlq_trace_begin": (i32, [i32]),
            "hlq_debug_reference_gemm": (i32, [i32, P, P, i64, i64, i64, P, P]),
            "hlq_debug_tc_gemm": (i32, [i32, P, i64, P, i64, i64, i64, i64, i32,
                                        i32, i32, P, P, sz, P]),
            "hlq_debug_tc_gemm_ws_bytes": (sz, [i64, i64]),
            "hlq_linear_backward_gx_noalloc": (i32, [P, P, i32, i64, i64, i64, i32,
                                                     i32, i32, i32, u64, P, P]),
            "hlq_noalloc_scratch_bytes": (sz, []),
            "hlq_linear_backward": (i32, [P, P, P, P, i32, i64, i64, i64, i32, i32,
                                          i32, i32, i32, i32, u64, P, P, P, sz, P]),
            "hlq_linear_backward_fused": (i32, [P, P, P, P, i32, i64, i64, i64, i32, i32,
                                          i32, i32, i32, i32, u64, P, P, P, sz, P]),
            "hlq_layer_step_host": (i32, [P, P, P, i32, i64, i64, i64, i32, i32, i32,
                                          i32, i32, i32, u64, P, P, P, P, i64, P, sz, P]),
            "hlq_layer_step_host_workspace_bytes": (sz, [i32, i64, i64, i64, i32, i32]),
            "hlq_select_gy_granularity": (i32, [P, i32, i64, i64, i32, ctypes.c_double,
                                                P, P, P, sz, P]),
            "hlq_ablation_gw_hq": (i32, [P, P, i32, i64, i64, i64, i32, i32, u64, P, P, P,
                                         sz, P]),
            "hlq_debug_gemm_plan": (i32, [i64, i64, i64, i32, i32, P, P, P, P, P, P, P]),
            "hlq_debug_wait_timeout": (i32, [u64, P, P]),
            "hlq_layer_step": (i32, [P, P, P, i32, i64, i64, i64, i32, i32, i32, i32, i32,
                                     i32, u64, P, P, P, P, P, sz, P]),
            "hlq_ablation_gx_hla": (i32, [P, P, i32, i64, i64, i64, i32, i32, P, P, P, sz,
                                          P]),
            "hlq_trace_end": (i32, [P]),
            "hlq_trace_get": (i32, [i32, P, P]),
            "hlq_trace_free": (i32, []),
            "hlq_set_gw_operands": (i32, [i32]),
            "hlq_get_gw_operands": (i32, []),
            "hlq_debug_serialize_branches": (i32, [i32]),
            "hlq_layer_norm": (i32, [P, i64, P, i64, i32, P, P, i32, i64, i64, f32, P, i64,
                                     i32, P, i64, P, P, P]),
            "hlq_layer_norm_backward": (i32, [P, i64, i32, P, i64, i32, P, P, P, i32, P, i64,
                                              i64, i64, P, i64, i32, P, P, P, sz, P]),
            "hlq_layer_norm_backward_workspace_bytes": (sz, [i64, i64]),
            "hlq_token_logprobs": (i32, [P, i64, i32, P, i64, i64, f32, P, P, P]),
            "hlq_policy_loss": (i32, [P, i64, i32, P, P, P, P, P, i64, i64, f32, f32, f32,
                                      f32, f32, P, P, P, i64, P, sz, P]),
            "hlq_policy_loss_workspace_bytes": (sz, [i64, i64]),
            "hlq_clip_grad_norm": (i32, [i64, P, P, P, P, P, f32, P, P, sz, P]),
            "hlq_clip_grad_norm_workspace_bytes": (sz, [i64]),
            "hlq_attention": (i32, [P, P, P, i32, i64, i64, i64, i64, i64, P, P, i64, i32, f32, P,
                                    P, P]),
            "hlq_attention_backward": (i32, [P, i32, P, P, P, P, i32, P, i64, i64, i64, i64, i64,
                                             P, P, i64, i32, f32, P, P, P, i32, P, sz, P]),
            "hlq_attention_backward_workspace_bytes": (sz, [i64, i64, i64, i32, i32]),
            "hlq_dropout": (i32, [P, i64, i32, P, i64, i64, i64, ctypes.c_double, u64, P, P, i64,
                                  i32, P]),
            "hlq_status_string": (ctypes.c_char_p, [i32]),
            "hlq_version": (i32, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
        return _lib


def status_string(status: int) -> str:
    return lib().hlq_status_string(int(status)).decode()


hlq_status_string = status_string


def _check(rc: int, what: str):
    if rc != 0:
        raise HLQError(rc, what)


# ----------------------------------------------------------------------------
# torch marshalling
# ----------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}: use bfloat16 or float32")


def _need_cuda_contig(*ts, current_device=None):
    """Contiguous CUDA tensors, all on the current device (the library
    launches on the current device and stream)."""
    index = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")
        if index is None:
            index = t.device.index
        elif t.device.index != index:
            raise ValueError(f"tensors must be on one device (cuda:{index} and "
                             f"cuda:{t.device.index})")
    if index is not None:
        cur = _torch().cuda.current_device() if current_device is None else current_device
        if index != cur:
            raise ValueError(f"tensors are on cuda:{index} but cuda:{cur} is current; "
                             "make their device current first")


def _need_buf(t, shape, dtype, index, what):
    """A caller-supplied output or buffer: a contiguous CUDA tensor on device
    `index` (the inputs' device) with exactly `shape` (None: any shape) and
    one of the dtypes `dtype`.  The kernels write through these pointers, so
    a wrong device, size or type is refused here rather than written past."""
    if not getattr(t, "is_cuda", False) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor")
    if t.device.index != index:
        raise ValueError(f"{what} is on cuda:{t.device.index}, the inputs on cuda:{index}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    dts = dtype if isinstance(dtype, tuple) else (dtype,)
    if t.dtype not in dts:
        raise ValueError(f"{what} must be of dtype {' or '.join(map(str, dts))}, "
                         f"not {t.dtype}")


def _ws_bytes(ws, index):
    """Size in bytes of a caller-supplied workspace (any dtype), after the
    same device and contiguity checks as an output."""
    if not getattr(ws, "is_cuda", False) or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous CUDA tensor")
    if ws.device.index != index:
        raise ValueError(f"ws is on cuda:{ws.device.index}, the inputs on cuda:{index}")
    return int(ws.numel()) * int(ws.element_size())


def hlq_workspace_bytes(op: int, T: int, Cin: int, Cout: int, block: int = 16,
                        rank: int = 8) -> int:
    return int(lib().hlq_workspace_bytes(op, T, Cin, Cout, block, rank))


def workspace(op, T, Cin, Cout, block=16, rank=8, device=None):
    torch = _torch()
    n = hlq_workspace_bytes(op, T, Cin, Cout, block, rank)
    return torch.empty(max(n, 256), dtype=torch.uint8,
                       device=device or torch.cuda.current_device())


def _xbar_fmt(xbar_bits: int, per_channel: bool) -> int:
    """Format word of the stored activation: code bits, plus the per-channel
    flag."""
    return int(xbar_bits) | (XBAR_PER_CHANNEL if per_channel else 0)


def _check_xbar_scale(xbar_scale, Cin: int, per_channel: bool):
    need = Cin if per_channel else 1
    if xbar_scale.dtype != _torch().float32 or xbar_scale.numel() != need:
        raise ValueError(f"xbar_scale must hold {need} fp32 value(s)")


def xbar_shape(T: int, Cin: int, rank: int = 8, xbar_bits: int = 8):
    """Shape of the ACBP buffer: [Cin, T'] int8 codes, or [Cin, T'/2] bytes
    of packed int4 codes."""
    Tp = T // 16 * rank
    return (Cin, Tp if xbar_bits == 8 else Tp // 2)


def _check_xbar(xbar, xbar_scale, T: int, Cin: int, rank: int, xbar_bits: int,
                per_channel: bool, index: int):
    """The ACBP buffer and its scales as the library reads or writes them:
    one-byte codes of exactly xbar_shape(...), fp32 scales [1] or [Cin]."""
    torch = _torch()
    _need_buf(xbar, xbar_shape(T, Cin, rank, xbar_bits), (torch.int8, torch.uint8), index,
              "xbar")
    _need_buf(xbar_scale, None, torch.float32, index, "xbar_scale")
    _check_xbar_scale(xbar_scale, Cin, per_channel)


def hlq_compress_activation(x, rank: int = 8, block: int = 16, out=None,
                            scale=None, ws=None, xbar_bits: int = 8, stream=None,
                            xbar_per_channel: bool = False):
    """ACBP: x [T, Cin] -> (codes, fp32 scale [1], or [Cin] with
    xbar_per_channel); codes are int8 [Cin, T*rank/16] (xbar_bits 8) or uint8
    [Cin, T*rank/32] holding two int4 codes per byte (xbar_bits 4)."""
    torch = _torch()
    _need_cuda_contig(x)
    T, Cin = x.shape
    dev = x.device
    if out is None:
        out = torch.empty(xbar_shape(T, Cin, rank, xbar_bits),
                          dtype=torch.int8 if xbar_bits == 8 else torch.uint8,
                          device=dev)
    if scale is None:
        scale = torch.empty(Cin if xbar_per_channel else 1, dtype=torch.float32,
                            device=dev)
    _check_xbar(out, scale, T, Cin, rank, xbar_bits, xbar_per_channel, dev.index)
    if ws is None:
        ws = workspace(OP_COMPRESS_ACTIVATION, T, Cin, 16, block, rank, dev)
    _check(lib().hlq_compress_activation(
        _ptr(x), _dtype_code(x), T, Cin, block, rank,
        _xbar_fmt(xbar_bits, xbar_per_channel), _ptr(out),
        _ptr(scale), _ptr(ws), _ws_bytes(ws, dev.index), _stream(stream)),
        "hlq_compress_activation")
    return out, scale


def hlq_linear_backward_gx(g_y, w, gran_gy: int = PER_TOKEN,
                           gran_w: int = PER_TENSOR, rnd: int = SR,
                           seed: int = 0, block: int = 16, out=None, ws=None,
                           stream=None):
    """g_x [T, Cin] (fp32) of y = x w^T from g_y [T, Cout] and w [Cout, Cin]."""
    torch = _torch()
    _need_cuda_contig(g_y, w)
    T, Cout = g_y.shape
    Cout2, Cin = w.shape
    if Cout2 != Cout or g_y.dtype != w.dtype:
        raise ValueError("shape/dtype mismatch between g_y and w")
    dev = g_y.device
    if out is None:
        out = torch.empty((T, Cin), dtype=torch.float32, device=dev)
    _need_buf(out, (T, Cin), torch.float32, dev.index, "out")
    if ws is None:
        ws = workspace(OP_BACKWARD_GX, T, Cin, Cout, block, 16, dev)
    _check(lib().hlq_linear_backward_gx(
        _ptr(g_y), _ptr(w), _dtype_code(g_y), T, Cin, Cout, block, gran_gy,
        gran_w, rnd, seed, _ptr(out), _ptr(ws), _ws_bytes(ws, dev.index), _stream(stream)),
        "hlq_linear_backward_gx")
    return out


def hlq_linear_backward_gw(g_y, xbar, xbar_scale, rank: int = 8,
                           block: int = 16, out=None, ws=None, xbar_bits: int = 8,
                           stream=None, xbar_per_channel: bool = False):
    """g_w [Cout, Cin] (fp32) from g_y [T, Cout] and the ACBP buffer."""
    torch = _torch()
    _need_cuda_contig(g_y, xbar, xbar_scale)
    T, Cout = g_y.shape
    Cin = xbar.shape[0]
    dev = g_y.device
    _check_xbar(xbar, xbar_scale, T, Cin, rank, xbar_bits, xbar_per_channel, dev.index)
    if out is None:
        out = torch.empty((Cout, Cin), dtype=torch.float32, device=dev)
    _need_buf(out, (Cout, Cin), torch.float32, dev.index, "out")
    if ws is None:
        ws = workspace(OP_BACKWARD_GW, T, Cin, Cout, block, rank, dev)
    _check(lib().hlq_linear_backward_gw(
        _ptr(g_y), _dtype_code(g_y), _ptr(xbar), _ptr(xbar_scale), T, Cin,
        Cout, block, rank, _xbar_fmt(xbar_bits, xbar_per_channel), _ptr(out), _ptr(ws),
        _ws_bytes(ws, dev.index), _stream(stream)),
        "hlq_linear_backward_gw")
    return out


def hlq_linear_backward_gx_noalloc(g_y, w, gran_gy: int = PER_TOKEN,
                                   gran_w: int = PER_TENSOR, rnd: int = SR,
                                   seed: int = 0, block: int = 16, out=None,
                                   stream=None):
    """hlq_linear_backward_gx without a workspace: for callers that cannot
    allocate device memory, the library uses its own fixed scratch array
    (see include/hlq.h for the size limit and the sharing rules).  `out`
    lets such callers pass a preallocated g_x as well."""
    torch = _torch()
    _need_cuda_contig(g_y, w)
    T, Cout = g_y.shape
    Cout2, Cin = w.shape
    if Cout2 != Cout or g_y.dtype != w.dtype:
        raise ValueError("shape/dtype mismatch between g_y and w")
    if out is None:
        out = torch.empty((T, Cin), dtype=torch.float32, device=g_y.device)
    _need_buf(out, (T, Cin), torch.float32, g_y.device.index, "out")
    _check(lib().hlq_linear_backward_gx_noalloc(
        _ptr(g_y), _ptr(w), _dtype_code(g_y), T, Cin, Cout, block, gran_gy,
        gran_w, rnd, seed, _ptr(out), _stream(stream)),
        "hlq_linear_backward_gx_noalloc")
    return out


def hlq_linear_backward(g_y, w, xbar, xbar_scale, rank: int = 8,
                        gran_gy: int = PER_TOKEN, gran_w: int = PER_TENSOR,
                        rnd: int = SR, seed: int = 0, block: int = 16,
                        out_gx=None, out_gw=None, ws=None, xbar_bits: int = 8,
                        stream=None, xbar_per_channel: bool = False,
                        fused_gy: bool = False):
    """Both gradients of the layer, the g_x and g_w branches overlapped on
    the GPU: returns (g_x [T, Cin], g_w [Cout, Cin]) fp32.  fused_gy: one
    fused reader of g_y for both paths (hlq_linear_backward_fused; same
    bits, workspace of OP_BACKWARD_FUSED)."""
    torch = _torch()
    _need_cuda_contig(g_y, w, xbar, xbar_scale)
    T, Cout = g_y.shape
    Cin = w.shape[1]
    if w.shape[0] != Cout or g_y.dtype != w.dtype or xbar.shape[0] != Cin:
        raise ValueError("shape/dtype mismatch between g_y, w and xbar")
    dev = g_y.device
    _check_xbar(xbar, xbar_scale, T, Cin, rank, xbar_bits, xbar_per_channel, dev.index)
    if out_gx is None:
        out_gx = torch.empty((T, Cin), dtype=torch.float32, device=dev)
    if out_gw is None:
        out_gw = torch.empty((Cout, Cin), dtype=torch.float32, device=dev)
    _need_buf(out_gx, (T, Cin), torch.float32, dev.index, "out_gx")
    _need_buf(out_gw, (Cout, Cin), torch.float32, dev.index, "out_gw")
    if ws is None:
        ws = workspace(OP_BACKWARD_FUSED if fused_gy else OP_BACKWARD, T, Cin, Cout, block,
                       rank, dev)
    fn = lib().hlq_linear_backward_fused if fused_gy else lib().hlq_linear_backward
    _check(fn(
        _ptr(g_y), _ptr(w), _ptr(xbar), _ptr(xbar_scale), _dtype_code(g_y), T,
        Cin, Cout, block, rank, _xbar_fmt(xbar_bits, xbar_per_channel), gran_gy,
        gran_w, rnd, seed, _ptr(out_gx),
        _ptr(out_gw), _ptr(ws), _ws_bytes(ws, dev.index), _stream(stream)),
        "hlq_linear_backward_fused" if fused_gy else "hlq_linear_backward")
    return out_gx, out_gw


def hlq_layer_step(x, g_y, w, rank: int = 8, gran_gy: int = PER_TOKEN,
                   gran_w: int = PER_TENSOR, rnd: int = SR, seed: int = 0, block: int = 16,
                   out_gx=None, out_gw=None, xbar=None, xbar_scale=None, ws=None,
                   xbar_bits: int = 8, xbar_per_channel: bool = False, stream=None):
    """The ACBP compression of x and both gradients in one call (the
    compression overlaps the g_x branch): returns (g_x, g_w, xbar,
    xbar_scale)."""
    torch = _torch()
    _need_cuda_contig(x, g_y, w)
    T, Cout = g_y.shape
    Cin = w.shape[1]
    if w.shape[0] != Cout or tuple(x.shape) != (T, Cin) or not (x.dtype == g_y.dtype == w.dtype):
        raise ValueError("shape/dtype mismatch between x, g_y and w")
    dev = g_y.device
    if out_gx is None:
        out_gx = torch.empty((T, Cin), dtype=torch.float32, device=dev)
    if out_gw is None:
        out_gw = torch.empty((Cout, Cin), dtype=torch.float32, device=dev)
    if xbar is None:
        xbar = torch.empty(xbar_shape(T, Cin, rank, xbar_bits),
                           dtype=torch.int8 if xbar_bits == 8 else torch.uint8, device=dev)
    if xbar_scale is None:
        xbar_scale = torch.empty(Cin if xbar_per_channel else 1, dtype=torch.float32,
                                 device=dev)
    _need_buf(out_gx, (T, Cin), torch.float32, dev.index, "out_gx")
    _need_buf(out_gw, (Cout, Cin), torch.float32, dev.index, "out_gw")
    _check_xbar(xbar, xbar_scale, T, Cin, rank, xbar_bits, xbar_per_channel, dev.index)
    if ws is None:
        ws = workspace(OP_LAYER_STEP, T, Cin, Cout, block, rank, dev)
    _check(lib().hlq_layer_step(
        _ptr(x), _ptr(g_y), _ptr(w), _dtype_code(g_y), T, Cin, Cout, block, rank,
        _xbar_fmt(xbar_bits, xbar_per_channel), gran_gy, gran_w, rnd, seed, _ptr(out_gx),
        _ptr(out_gw), _ptr(xbar), _ptr(xbar_scale), _ptr(ws), _ws_bytes(ws, dev.index),
        _stream(stream)),
        "hlq_layer_step")
    return out_gx, out_gw, xbar, xbar_scale


def _need_cpu_contig(*ts):
    for t in ts:
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError("host tensors must be contiguous CPU tensors")


def _need_host_out(t, shape, what):
    """A caller-supplied host output: a contiguous fp32 CPU tensor of exactly
    `shape` (the library's copies write its whole extent)."""
    _need_cpu_contig(t)
    if tuple(t.shape) != tuple(shape) or t.dtype != _torch().float32:
        raise ValueError(f"{what} must be a float32 CPU tensor of shape {tuple(shape)}")


def hlq_layer_step_host_workspace_bytes(dtype_code: int, T: int, Cin: int, Cout: int,
                                        block: int = 16, rank: int = 8) -> int:
    return int(lib().hlq_layer_step_host_workspace_bytes(dtype_code, T, Cin, Cout, block,
                                                         rank))


def hlq_layer_step_host(x, g_y, w, xbar, xbar_scale, rank: int = 8,
                        gran_gy: int = PER_TOKEN, gran_w: int = PER_TENSOR,
                        rnd: int = SR, seed: int = 0, block: int = 16,
                        out_gx=None, out_gw=None, ws=None, chunk_tokens: int = 0,
                        xbar_bits: int = 8, stream=None, xbar_per_channel: bool = False):
    """One layer step from host tensors (x, g_y, w on the CPU, pinned for
    speed): compresses x into the device buffers xbar / xbar_scale and
    returns host (g_x, g_w) fp32.  Asynchronous on `stream`: synchronize it
    before reading the results."""
    torch = _torch()
    _need_cpu_contig(x, g_y, w, out_gx, out_gw)
    _need_cuda_contig(xbar, xbar_scale)
    T, Cout = g_y.shape
    Cin = w.shape[1]
    if w.shape[0] != Cout or tuple(x.shape) != (T, Cin) or not (x.dtype == g_y.dtype == w.dtype):
        raise ValueError("shape/dtype mismatch between x, g_y and w")
    index = xbar.device.index
    _check_xbar(xbar, xbar_scale, T, Cin, rank, xbar_bits, xbar_per_channel, index)
    if out_gx is None:
        out_gx = torch.empty((T, Cin), dtype=torch.float32).pin_memory()
    if out_gw is None:
        out_gw = torch.empty((Cout, Cin), dtype=torch.float32).pin_memory()
    _need_host_out(out_gx, (T, Cin), "out_gx")
    _need_host_out(out_gw, (Cout, Cin), "out_gw")
    dt = _dtype_code(g_y)
    if ws is None:
        n = hlq_layer_step_host_workspace_bytes(dt, T, Cin, Cout, block, rank)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=xbar.device)
    _check(lib().hlq_layer_step_host(
        _ptr(x), _ptr(g_y), _ptr(w), dt, T, Cin, Cout, block, rank,
        _xbar_fmt(xbar_bits, xbar_per_channel), gran_gy, gran_w,
        rnd, seed, _ptr(out_gx), _ptr(out_gw), _ptr(xbar), _ptr(xbar_scale),
        chunk_tokens, _ptr(ws), _ws_bytes(ws, index), _stream(stream)),
        "hlq_layer_step_host")
    return out_gx, out_gw


def hlq_select_gy_granularity(g_y, threshold: float = 1.5, block: int = 16,
                              stream=None, mse=None, choice=None, ws=None):
    """Layer-wise quantizer selection on a calibration sample g_y [T, Cout]:
    returns device tensors (mse [2] fp64: per tensor, per token; choice [1]
    int32: PER_TOKEN or PER_TENSOR); mse / choice / ws may be preallocated."""
    torch = _torch()
    _need_cuda_contig(g_y)
    T, Cout = g_y.shape
    dev = g_y.device
    if mse is None:
        mse = torch.empty(2, dtype=torch.float64, device=dev)
    if choice is None:
        choice = torch.empty(1, dtype=torch.int32, device=dev)
    _need_buf(mse, (2,), torch.float64, dev.index, "mse")
    _need_buf(choice, (1,), torch.int32, dev.index, "choice")
    if ws is None:
        ws = workspace(OP_SELECT_GRANULARITY, T, 16, Cout, block, 8, dev)
    _check(lib().hlq_select_gy_granularity(
        _ptr(g_y), _dtype_code(g_y), T, Cout, block, float(threshold), _ptr(mse),
        _ptr(choice), _ptr(ws), _ws_bytes(ws, dev.index), _stream(stream)),
        "hlq_select_gy_granularity")
    return mse, choice


def hlq_ablation_gw_hq(g_y, x, rnd: int = SR, seed: int = 0, block: int = 16,
                       with_acc: bool = False, stream=None, out=None, ws=None):
    """g_w [Cout, Cin] through HQ along tokens (the ablation of the g_w path);
    with_acc also returns the int32 accumulator."""
    torch = _torch()
    _need_cuda_contig(g_y, x)
    T, Cout = g_y.shape
    Cin = x.shape[1]
    if x.shape[0] != T or x.dtype != g_y.dtype:
        raise ValueError("shape/dtype mismatch between g_y and x")
    dev = g_y.device
    gw = (torch.empty((Cout, Cin), dtype=torch.float32, device=dev)
          if out is None else out)
    _need_buf(gw, (Cout, Cin), torch.float32, dev.index, "out")
    acc = (torch.empty((Cout, Cin), dtype=torch.int32, device=dev)
           if with_acc else None)
    if ws is None:
        ws = workspace(OP_ABLATION_GW_HQ, T, Cin, Cout, block, 8, dev)
    _check(lib().hlq_ablation_gw_hq(
        _ptr(g_y), _ptr(x), _dtype_code(g_y), T, Cin, Cout, block, rnd, seed, _ptr(gw),
        _ptr(acc), _ptr(ws), _ws_bytes(ws, dev.index), _stream(stream)),
        "hlq_ablation_gw_hq")
    return (gw, acc) if with_acc else gw


def hlq_ablation_gx_hla(g_y, w, rank: int = 8, block: int = 16, with_acc: bool = False,
                        stream=None, out=None, ws=None):
    """g_x [T, Cin] through HLA along Cout with int8 codes (the ablation of
    the g_x path); with_acc also returns the int32 accumulator."""
    torch = _torch()
    _need_cuda_contig(g_y, w)
    T, Cout = g_y.shape
    Cin = w.shape[1]
    if w.shape[0] != Cout or w.dtype != g_y.dtype:
        raise ValueError("shape/dtype mismatch between g_y and w")
    dev = g_y.device
    gx = (torch.empty((T, Cin), dtype=torch.float32, device=dev)
          if out is None else out)
    _need_buf(gx, (T, Cin), torch.float32, dev.index, "out")
    acc = (torch.empty((T, Cin), dtype=torch.int32, device=dev)
           if with_acc else None)
    if ws is None:
        ws = workspace(OP_ABLATION_GX_HLA, T, Cin, Cout, block, rank, dev)
    _check(lib().hlq_ablation_gx_hla(
        _ptr(g_y), _ptr(w), _dtype_code(g_y), T, Cin, Cout, block, rank, _ptr(gx),
        _ptr(acc), _ptr(ws), _ws_bytes(ws, dev.index), _stream(stream)),
        "hlq_ablation_gx_hla")
    return (gx, acc) if with_acc else gx


# ----------------------------------------------------------------------------
# Around the layer in a training step
# ----------------------------------------------------------------------------

_ext = None


class _NoExt:
    """Where the extension is not built: nothing is taken at once."""

    def __getattr__(self, name):
        return lambda *args: NotImplemented


def _load_ext():
    """The extension module that checks, allocates and calls in one step: what
    it does not take at once, or the library refuses, it answers with
    NotImplemented, and the entry point goes on in Python."""
    global _ext
    _torch()
    from .build import ext_path
    path = ext_path()
    if not os.path.exists(path):
        warnings.warn(f"the binding's extension is not built for this torch ({path} missing; run "
                      "`python -m hadamard_precision_backprop_gb300.build`): calls of the operators "
                      "around the layer cost the host some 20 us more", RuntimeWarning)
        _ext = _NoExt()
        return _ext
    spec = importlib.util.spec_from_file_location("_hlq_torch", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    _ext = module
    return _ext


def _on_stream(call, args):
    """`call` with the keyword arguments `args`, their stream current: what it
    allocates (outputs, workspace) then belongs to the stream that uses it."""
    stream = args.pop("stream")
    with _torch().cuda.stream(stream):
        return call(**args)


def _raw_stream(index):
    """torch's current stream of device `index`, as the library takes it."""
    return _torch()._C._cuda_getCurrentRawStream(index)


_dtype_codes = {}


def _code(dtype):
    code = _dtype_codes.get(dtype)
    if code is None:
        torch = _torch()
        _dtype_codes.update({torch.float32: F32, torch.bfloat16: BF16})
        code = _dtype_codes.get(dtype)
        if code is None:
            raise TypeError(f"unsupported dtype {dtype}: use bfloat16 or float32")
    return code


def _rows(t, what, index=None, shape=None, dtype=None):
    """Row stride, dtype code and address of a [rows, columns] CUDA tensor
    whose rows are contiguous (any row stride, 0 for a repeated row), on
    device `index`, of `shape` and of `dtype` where these are given."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if shape is None:
        if t.dim() != 2:
            raise ValueError(f"{what} must have shape [rows, columns], not {tuple(t.shape)}")
    elif t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    ld, step = t.stride()
    if step != 1 and t.shape[1] > 1:
        raise ValueError(f"the rows of {what} must be contiguous")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{what} is on cuda:{t.get_device()}, the inputs on cuda:{index}")
    own = t.dtype
    if dtype is not None and own != dtype:
        raise ValueError(f"{what} must be of dtype {dtype}, not {own}")
    return ld, _code(own), t.data_ptr()


def _new_rows(t, cols):
    """The same of an output that the call has just allocated."""
    return cols, _code(t.dtype), t.data_ptr()


def _vector(t, what, n, index, dtype=None):
    """Address of a contiguous CUDA tensor [n] (None: a null pointer)."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{what} is on cuda:{t.get_device()}, the inputs on cuda:{index}")
    if t.shape != (n,):
        raise ValueError(f"{what} must have shape ({n},), not {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be of dtype {dtype}, not {t.dtype}")
    return t.data_ptr()


def _out_vector(t, what, n, index, device):
    """An fp32 output [n], the caller's or a new one, and its address."""
    if t is None:
        t = _torch().empty(n, dtype=_torch().float32, device=device)
        return t, t.data_ptr()
    return t, _vector(t, what, n, index, _torch().float32)


def _workspace(ws, n, index, device):
    """A workspace of n bytes, the caller's or a new one: the tensor (which
    must outlive the call), its address and its size."""
    if ws is None:
        ws = _torch().empty(n, dtype=_torch().uint8, device=device)
        return ws, ws.data_ptr(), n
    return ws, ws.data_ptr(), _ws_bytes(ws, index)


def _need_current(index):
    cur = _torch().cuda.current_device()
    if index != cur:
        raise ValueError(f"tensors are on cuda:{index} but cuda:{cur} is current; "
                         "make their device current first")


def hlq_layer_norm(x, weight=None, bias=None, eps: float = 1e-5, residual=None,
                   out_dtype=None, out=None, h=None, mean=None, rstd=None,
                   with_stats: bool = True, stream=None):
    """Layer norm of x [T, C] (of h = x + residual where one is given): returns
    (y, mean, rstd), or (y, mean, rstd, h) with a residual.  y has `out_dtype`
    (default: x's); mean and rstd are fp32 [T], for the backward pass, and None
    with with_stats=False.  x, residual, out and h may have any row stride."""
    if stream is not None:
        return _on_stream(hlq_layer_norm, locals())
    if out is None and h is None and mean is None and rstd is None:
        got = (_ext or _load_ext()).layer_norm(x, weight, bias, eps, residual, out_dtype,
                                               with_stats)
        if got is not NotImplemented:
            return got
    torch = _torch()
    ldx, dt, px = _rows(x, "x")
    shape, index, device = x.shape, x.get_device(), x.device
    _need_current(index)
    T, C = shape
    w_dt = F32
    if weight is not None:
        w_dt = _code(weight.dtype)
    elif bias is not None:
        w_dt = _code(bias.dtype)
    pw = _vector(weight, "weight", C, index)
    pb = _vector(bias, "bias", C, index)
    if pw is not None and pb is not None and weight.dtype != bias.dtype:
        raise ValueError("weight and bias must have one dtype")
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or x.dtype, device=device)
        ldy, y_dt, py = _new_rows(out, C)
    else:
        ldy, y_dt, py = _rows(out, "out", index, shape, out_dtype)
    ldr = ldh = 0
    pr = ph = pm = ps = None
    if residual is not None:
        ldr, _, pr = _rows(residual, "residual", index, shape, x.dtype)
        if h is None:
            h = torch.empty(shape, dtype=x.dtype, device=device)
        ldh, _, ph = _rows(h, "h", index, shape, x.dtype)
    elif h is not None:
        raise ValueError("h is written only with a residual")
    if with_stats:
        mean, pm = _out_vector(mean, "mean", T, index, device)
        rstd, ps = _out_vector(rstd, "rstd", T, index, device)
    elif mean is not None or rstd is not None:
        raise ValueError("mean and rstd are written only with with_stats")
    rc = lib().hlq_layer_norm(px, ldx, pr, ldr, dt, pw, pb, w_dt, T, C, eps, py, ldy, y_dt, ph,
                              ldh, pm, ps, _raw_stream(index))
    _check(rc, "hlq_layer_norm")
    return (out, mean, rstd) if residual is None else (out, mean, rstd, h)


def hlq_layer_norm_backward(g_y, x, mean, rstd, weight=None, g_residual=None, out_dtype=None,
                            out=None, g_weight=None, g_bias=None,
                            with_weight_grads: bool = True, ws=None, stream=None):
    """Backward pass of hlq_layer_norm: g_y [T, C] (bf16 or fp32, whatever x's
    type), x the normalised input (h where there was a residual) and its mean
    and rstd.  Returns (g_x, g_weight, g_bias): g_x of `out_dtype` (default:
    x's), with g_residual (of that type) added; g_weight and g_bias fp32 [C],
    None with with_weight_grads=False."""
    if stream is not None:
        return _on_stream(hlq_layer_norm_backward, locals())
    if out is None and g_weight is None and g_bias is None and ws is None:
        got = (_ext or _load_ext()).layer_norm_backward(g_y, x, mean, rstd, weight, g_residual,
                                                        out_dtype, with_weight_grads)
        if got is not NotImplemented:
            return got
    torch = _torch()
    f32 = torch.float32
    ldx, x_dt, px = _rows(x, "x")
    shape, index, device = x.shape, x.get_device(), x.device
    _need_current(index)
    T, C = shape
    ldgy, gy_dt, pgy = _rows(g_y, "g_y", index, shape)
    pm = _vector(mean, "mean", T, index, f32)
    ps = _vector(rstd, "rstd", T, index, f32)
    pw = _vector(weight, "weight", C, index)
    w_dt = F32 if weight is None else _code(weight.dtype)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or x.dtype, device=device)
        ldgx, gx_dt, pgx = _new_rows(out, C)
    else:
        ldgx, gx_dt, pgx = _rows(out, "out", index, shape, out_dtype)
    ldgr, pgr = 0, None
    if g_residual is not None:
        ldgr, _, pgr = _rows(g_residual, "g_residual", index, shape, out.dtype)
    pgw = pgb = pws = None
    n_ws = 0
    if with_weight_grads:
        g_weight, pgw = _out_vector(g_weight, "g_weight", C, index, device)
        g_bias, pgb = _out_vector(g_bias, "g_bias", C, index, device)
        if ws is None:
            n_ws = lib().hlq_layer_norm_backward_workspace_bytes(T, C)
        ws, pws, n_ws = _workspace(ws, n_ws, index, device)
    elif g_weight is not None or g_bias is not None:
        raise ValueError("g_weight and g_bias are written only with with_weight_grads")
    rc = lib().hlq_layer_norm_backward(pgy, ldgy, gy_dt, px, ldx, x_dt, pm, ps, pw, w_dt, pgr,
                                       ldgr, T, C, pgx, ldgx, gx_dt, pgw, pgb, pws, n_ws,
                                       _raw_stream(index))
    _check(rc, "hlq_layer_norm_backward")
    return out, g_weight, g_bias


def hlq_token_logprobs(logits, targets, scale: float = 1.0, logp=None, lse=None, stream=None):
    """log softmax(scale * logits) [T, V] at targets (int64 [T]) and the rows'
    log-sum-exp: (logp, lse), fp32 [T]."""
    if stream is not None:
        return _on_stream(hlq_token_logprobs, locals())
    if logp is None and lse is None:
        got = (_ext or _load_ext()).token_logprobs(logits, targets, scale)
        if got is not NotImplemented:
            return got
    ld, dt, pl = _rows(logits, "logits")
    T, V = logits.shape
    index, device = logits.get_device(), logits.device
    _need_current(index)
    pt = _vector(targets, "targets", T, index, _torch().int64)
    logp, pp = _out_vector(logp, "logp", T, index, device)
    lse, ps = _out_vector(lse, "lse", T, index, device)
    rc = lib().hlq_token_logprobs(pl, ld, dt, pt, T, V, scale, pp, ps, _raw_stream(index))
    _check(rc, "hlq_token_logprobs")
    return logp, lse


def hlq_policy_loss(logits, actions, old_logp, advantages, weights, ref_logp=None,
                    clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0,
                    scale: float = 1.0, grad_scale: float = 1.0, with_grad: bool = True,
                    stats=None, logp=None, out=None, ws=None, stream=None):
    """Clipped policy loss with a KL term to a reference (see include/hlq.h for
    the formulas) over logits [T, V], and its gradient: (stats, logp, g).
    stats fp32 [4]: loss, policy term, KL term, clipped share of the weights;
    logp fp32 [T]; g [T, V] in the logits' dtype, grad_scale times the gradient
    of the loss (None with with_grad=False; out=logits overwrites them).
    actions int64 [T]; old_logp, advantages, weights, ref_logp fp32 [T]; a row
    of weight 0 takes no part and is not read."""
    if stream is not None:
        return _on_stream(hlq_policy_loss, locals())
    if stats is None and logp is None and out is None and ws is None:
        got = (_ext or _load_ext()).policy_loss(logits, actions, old_logp, advantages, weights,
                                                ref_logp, clip_low, clip_high, kl_coef, scale,
                                                grad_scale, with_grad)
        if got is not NotImplemented:
            return got
    torch = _torch()
    f32 = torch.float32
    ld, dt, pl = _rows(logits, "logits")
    shape, index, device = logits.shape, logits.get_device(), logits.device
    _need_current(index)
    T, V = shape
    pa = _vector(actions, "actions", T, index, torch.int64)
    po = _vector(old_logp, "old_logp", T, index, f32)
    pr = _vector(ref_logp, "ref_logp", T, index, f32)
    pv = _vector(advantages, "advantages", T, index, f32)
    pw = _vector(weights, "weights", T, index, f32)
    stats, ps = _out_vector(stats, "stats", 4, index, device)
    logp, pp = _out_vector(logp, "logp", T, index, device)
    ldg, pg = 0, None
    if with_grad:
        if out is None:
            out = torch.empty(shape, dtype=logits.dtype, device=device)
            ldg, _, pg = _new_rows(out, V)
        else:
            ldg, _, pg = _rows(out, "out", index, shape, logits.dtype)
    elif out is not None:
        raise ValueError("out is written only with with_grad")
    n_ws = lib().hlq_policy_loss_workspace_bytes(T, V) if ws is None else 0
    ws, pws, n_ws = _workspace(ws, n_ws, index, device)
    rc = lib().hlq_policy_loss(pl, ld, dt, pa, po, pr, pv, pw, T, V, scale, clip_low, clip_high,
                               kl_coef, grad_scale, ps, pp, pg, ldg, pws, n_ws,
                               _raw_stream(index))
    _check(rc, "hlq_policy_loss")
    return stats, logp, out


def _table(ts, what, index):
    """Addresses, dtype codes and element counts of contiguous tensors on
    device `index`, as the arrays the library takes."""
    if not all([t.is_contiguous() for t in ts]):
        raise ValueError(f"{what} must be contiguous CUDA tensors")
    if {t.get_device() for t in ts} - {index}:
        if not all([t.is_cuda for t in ts]):
            raise ValueError(f"{what} must be contiguous CUDA tensors")
        raise ValueError(f"{what} must be on one device")
    return (array.array("Q", [t.data_ptr() for t in ts]),
            array.array("i", [_code(t.dtype) for t in ts]),
            array.array("q", [t.numel() for t in ts]))


def hlq_clip_grad_norm(grads, max_norm: float, outs=None, norm_only: bool = False,
                       norm_coef=None, ws=None, stream=None):
    """Global norm of `grads` (contiguous bf16 / fp32 CUDA tensors of any
    shapes) and their clipping to max_norm: writes coef * g to `outs` (tensors
    of as many elements, bf16 or fp32), or over the gradients themselves by
    default, or nowhere with norm_only.  Returns fp32 [2]: norm, coef."""
    if stream is not None:
        return _on_stream(hlq_clip_grad_norm, locals())
    grads = list(grads)
    if norm_coef is None and ws is None:
        got = (_ext or _load_ext()).clip_grad_norm(grads, max_norm, outs, norm_only)
        if got is not NotImplemented:
            return got
    torch = _torch()
    n = len(grads)
    if norm_only and outs is not None:
        raise ValueError("norm_only writes no outs")
    if outs is not None:
        outs = list(outs)
        if len(outs) != n:
            raise ValueError(f"{len(outs)} outs for {n} gradients")
    index = grads[0].get_device() if n else torch.cuda.current_device()
    _need_current(index)
    g_ptr, g_dt, numels = _table(grads, "grads", index)
    o_ptr, o_dt = (None, None) if norm_only else (g_ptr, g_dt)
    if outs is not None:
        o_ptr, o_dt, o_numels = _table(outs, "outs", index)
        if o_numels != numels:
            raise ValueError("outs must have as many elements as the gradients")
    device = torch.device("cuda", index)
    norm_coef, pn = _out_vector(norm_coef, "norm_coef", 2, index, device)
    n_ws = lib().hlq_clip_grad_norm_workspace_bytes(n) if ws is None else 0
    ws, pws, n_ws = _workspace(ws, n_ws, index, device)
    at = lambda a: None if a is None else a.buffer_info()[0]  # noqa: E731
    rc = lib().hlq_clip_grad_norm(n, at(g_ptr), at(g_dt), at(o_ptr), at(o_dt), at(numels),
                                  max_norm, pn, pws, n_ws, _raw_stream(index))
    _check(rc, "hlq_clip_grad_norm")
    return norm_coef


class _Heads(ctypes.Structure):
    """hlq_heads: a [tokens, heads, D] tensor, its strides in elements."""
    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


def _heads(t, what, index=None, shape=None, dtype=None):
    """hlq_heads of a CUDA tensor [tokens, heads, D] whose heads are contiguous
    (any strides of tokens and heads), on device `index`, of `shape` and of
    `dtype` where these are given."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if shape is None:
        if t.dim() != 3:
            raise ValueError(f"{what} must have shape [tokens, heads, D], not {tuple(t.shape)}")
    elif t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    token, head, step = t.stride()
    if step != 1 and t.shape[2] > 1:
        raise ValueError(f"the heads of {what} must be contiguous")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{what} is on cuda:{t.get_device()}, the inputs on cuda:{index}")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be of dtype {dtype}, not {t.dtype}")
    return ctypes.byref(_Heads(t.data_ptr(), token, head))


def _sequences(seqs, seqs_k, batch, index):
    """Addresses of the offsets and the number of sequences."""
    if seqs is None:
        if seqs_k is not None:
            raise ValueError("seqs_k needs seqs")
        return None, None, int(batch)
    i32 = _torch().int32
    n = seqs.shape[0] if seqs.dim() == 1 else 0
    if n < 2:
        raise ValueError(f"seqs must have shape (batch + 1,), not {tuple(seqs.shape)}")
    if batch not in (1, n - 1):
        raise ValueError(f"seqs holds {n - 1} sequences, batch is {batch}")
    return (_vector(seqs, "seqs", n, index, i32), _vector(seqs_k, "seqs_k", n, index, i32), n - 1)


def _qkv(q, k, v):
    """What the attention calls have in common: the arguments, the device."""
    pq = _heads(q, "q")
    _code(q.dtype)
    index = q.get_device()
    _need_current(index)
    pk = _heads(k, "k", index, dtype=q.dtype)
    if k.shape[2] != q.shape[2]:
        raise ValueError(f"q has heads of {q.shape[2]}, k of {k.shape[2]}")
    if k.shape[1] < 1 or q.shape[1] % k.shape[1]:
        raise ValueError(f"the {k.shape[1]} heads of k must divide the {q.shape[1]} of q")
    return pq, pk, _heads(v, "v", index, k.shape, q.dtype), index


def hlq_attention(q, k, v, seqs=None, seqs_k=None, batch: int = 1, causal: bool = False,
                  scale=None, out=None, lse=None, stream=None):
    """Softmax attention over packed sequences: q [Tq, Hq, D], k and v [Tk, Hk,
    D] (bf16 or fp32, any token and head strides: parts of a qkv layer's output
    as they are; Hk divides Hq).  Returns (out [Tq, Hq, D], lse fp32 [Tq, Hq]).
    `batch` sequences of one length, or `seqs` int32 [batch + 1]: offsets of the
    sequences' queries (and keys; seqs_k where those have their own).  causal:
    the last query sees all keys, each before it one fewer.  scale: 1/sqrt(D) by
    default.  Rows of no sequence and queries that see nothing: 0, lse -inf."""
    if stream is not None:
        return _on_stream(hlq_attention, locals())
    if out is None and lse is None:
        got = (_ext or _load_ext()).attention(q, k, v, seqs, seqs_k, batch, causal, scale)
        if got is not NotImplemented:
            return got
    torch = _torch()
    pq, pk, pv, index = _qkv(q, k, v)
    Tq, Hq, D = q.shape
    ps, psk, batch = _sequences(seqs, seqs_k, batch, index)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    po = _heads(out, "out", index, q.shape, q.dtype)
    if lse is None:
        lse = torch.empty((Tq, Hq), dtype=torch.float32, device=q.device)
    _need_buf(lse, (Tq, Hq), torch.float32, index, "lse")
    scale = max(D, 1) ** -0.5 if scale is None else scale
    rc = lib().hlq_attention(pq, pk, pv, _code(q.dtype), Tq, k.shape[0], Hq, k.shape[1], D, ps, psk,
                             batch, 1 if causal else 0, scale, po, lse.data_ptr(),
                             _raw_stream(index))
    _check(rc, "hlq_attention")
    return out, lse


def hlq_attention_backward(g_out, q, k, v, out, lse, seqs=None, seqs_k=None, batch: int = 1,
                           causal: bool = False, scale=None, out_dtype=None, packed: bool = False,
                           g_q=None, g_k=None, g_v=None, ws=None, stream=None):
    """Backward pass of hlq_attention, from its inputs and outputs and g_out [Tq,
    Hq, D] (bf16 or fp32, whatever q's type): (g_q, g_k, g_v) of `out_dtype`
    (default: q's), or with packed=True (as many keys as queries) one tensor
    [T, Hq + 2 Hk, D] that holds them one after the other within each token: the
    gradient of a qkv layer's output."""
    if stream is not None:
        return _on_stream(hlq_attention_backward, locals())
    if g_q is None and g_k is None and g_v is None and ws is None:
        got = (_ext or _load_ext()).attention_backward(g_out, q, k, v, out, lse, seqs, seqs_k,
                                                       batch, causal, scale, out_dtype, packed)
        if got is not NotImplemented:
            return got
    torch = _torch()
    pq, pk, pv, index = _qkv(q, k, v)
    Tq, Hq, D = q.shape
    Tk, Hk, _ = k.shape
    pg = _heads(g_out, "g_out", index, q.shape)
    po = _heads(out, "out", index, q.shape, q.dtype)
    _need_buf(lse, (Tq, Hq), torch.float32, index, "lse")
    ps, psk, batch = _sequences(seqs, seqs_k, batch, index)
    g_all = None
    if packed:
        if g_q is not None or g_k is not None or g_v is not None:
            raise ValueError("packed allocates g_q, g_k and g_v itself")
        if Tq != Tk:
            raise ValueError(f"packed gradients need as many keys as queries, not {Tk} and {Tq}")
        g_all = torch.empty((Tq, Hq + 2 * Hk, D), dtype=out_dtype or q.dtype, device=q.device)
        g_q, g_k, g_v = g_all.split([Hq, Hk, Hk], 1)
    given = [t for t in (g_q, g_k, g_v) if t is not None]
    g_dtype = out_dtype or (given[0].dtype if given else q.dtype)
    if g_q is None:
        g_q = torch.empty(q.shape, dtype=g_dtype, device=q.device)
    if g_k is None:
        g_k = torch.empty(k.shape, dtype=g_dtype, device=q.device)
    if g_v is None:
        g_v = torch.empty(k.shape, dtype=g_dtype, device=q.device)
    pgq = _heads(g_q, "g_q", index, q.shape, g_dtype)
    pgk = _heads(g_k, "g_k", index, k.shape, g_dtype)
    pgv = _heads(g_v, "g_v", index, k.shape, g_dtype)
    dt, gout_dt = _code(q.dtype), _code(g_out.dtype)
    n_ws = 0
    if ws is None:
        n_ws = lib().hlq_attention_backward_workspace_bytes(Tq, Hq, D, dt, gout_dt)
    ws, pws, n_ws = _workspace(ws, n_ws, index, q.device)
    rc = lib().hlq_attention_backward(
        pg, gout_dt, pq, pk, pv, po, dt, lse.data_ptr(), Tq, Tk, Hq, Hk, D, ps, psk, batch,
        1 if causal else 0, max(D, 1) ** -0.5 if scale is None else scale, pgq, pgk, pgv,
        _code(g_dtype), pws, n_ws, _raw_stream(index))
    _check(rc, "hlq_attention_backward")
    return g_all if packed else (g_q, g_k, g_v)


def hlq_dropout(x, p: float, seed, residual=None, out_dtype=None, out=None, stream=None):
    """Dropout of x [T, C] with the residual added: each element kept with
    probability 1 - p (in steps of 2^-16) and divided by it.  The mask is drawn
    from `seed` (an int, or an int64 CUDA tensor of one element, which a
    captured graph reads anew at each replay) and the element's place alone, and
    is never stored: the backward pass is the same call on the gradient of y,
    without the residual.  y has `out_dtype` (default: residual's, or x's) and
    so has the residual."""
    if stream is not None:
        return _on_stream(hlq_dropout, locals())
    if out is None:
        got = (_ext or _load_ext()).dropout(x, p, seed, residual, out_dtype)
        if got is not NotImplemented:
            return got
    torch = _torch()
    ldx, x_dt, px = _rows(x, "x")
    shape, index, device = x.shape, x.get_device(), x.device
    _need_current(index)
    T, C = shape
    if out is None:
        dtype = out_dtype or (x.dtype if residual is None else residual.dtype)
        out = torch.empty(shape, dtype=dtype, device=device)
        ldy, y_dt, py = _new_rows(out, C)
    else:
        ldy, y_dt, py = _rows(out, "out", index, shape, out_dtype)
    ldr, pr = 0, None
    if residual is not None:
        ldr, _, pr = _rows(residual, "residual", index, shape, out.dtype)
    pd = None
    if isinstance(seed, torch.Tensor):
        if not seed.is_cuda or seed.get_device() != index or seed.numel() != 1 \
                or seed.dtype != torch.int64:
            raise ValueError(f"seed must be an int or an int64 tensor of one element on cuda:{index}")
        seed, pd = 0, seed.data_ptr()
    rc = lib().hlq_dropout(px, ldx, x_dt, pr, ldr, T, C, p, int(seed) & (2 ** 64 - 1), pd, py, ldy,
                           y_dt, _raw_stream(index))
    _check(rc, "hlq_dropout")
    return out


def hlq_debug_gx_parts(g_y, w, gran_gy=PER_TOKEN, gran_w=PER_TENSOR, rnd=SR,
                       seed=0, block=16, stream=None):
    """g_x plus its intermediates: dict(g_x, qgy, sgy, qw, sw, acc, and the
    codes as packed int4 bytes: qgy_packed [T, Cout/2], qw_packed [Cin,
    Cout/2])."""
    torch = _torch()
    _need_cuda_contig(g_y, w)
    T, Cout = g_y.shape
    Cin = w.shape[1]
    dev = g_y.device
    r = dict(
        g_x=torch.empty((T, Cin), dtype=torch.float32, device=dev),
        qgy=torch.empty((T, Cout), dtype=torch.int8, device=dev),
        sgy=torch.empty(T if gran_gy == PER_TOKEN else 1, dtype=torch.float32,
                        device=dev),
        qw=torch.empty((Cin, Cout), dtype=torch.int8, device=dev),
        sw=torch.empty(1, dtype=torch.float32, device=dev),
        acc=torch.empty((T, Cin), dtype=torch.int32, device=dev),
        qgy_packed=torch.empty((T, Cout // 2), dtype=torch.uint8, device=dev),
        qw_packed=torch.empty((Cin, Cout // 2), dtype=torch.uint8, device=dev),
    )
    ws = workspace(OP_BACKWARD_GX, T, Cin, Cout, block, 16, dev)
    _check(lib().hlq_debug_gx_parts(
        _ptr(g_y), _ptr(w), _dtype_code(g_y), T, Cin, Cout, block, gran_gy,
        gran_w, rnd, seed, _ptr(r["g_x"]), _ptr(ws), _ws_bytes(ws, dev.index),
        _ptr(r["qgy"]), _ptr(r["sgy"]), _ptr(r["qw"]), _ptr(r["sw"]),
        _ptr(r["acc"]), _ptr(r["qgy_packed"]), _ptr(r["qw_packed"]), _stream(stream)),
        "hlq_debug_gx_parts")
    return r


def hlq_debug_gw_parts(g_y, xbar, xbar_scale, rank=8, block=16, xbar_bits=8,
                       stream=None, xbar_per_channel=False):
    """g_w plus its intermediates: dict(g_w, qg, sg, acc)."""
    torch = _torch()
    _need_cuda_contig(g_y, xbar, xbar_scale)
    T, Cout = g_y.shape
    Cin = xbar.shape[0]
    _check_xbar_scale(xbar_scale, Cin, xbar_per_channel)
    Tp = T // 16 * rank
    dev = g_y.device
    r = dict(
        g_w=torch.empty((Cout, Cin), dtype=torch.float32, device=dev),
        qg=torch.empty((Cout, Tp), dtype=torch.int8, device=dev),
        sg=torch.empty(1, dtype=torch.float32, device=dev),
        acc=torch.empty((Cout, Cin), dtype=torch.int32, device=dev),
    )
    ws = workspace(OP_BACKWARD_GW, T, Cin, Cout, block, rank, dev)
    _check(lib().hlq_debug_gw_parts(
        _ptr(g_y), _dtype_code(g_y), _ptr(xbar), _ptr(xbar_scale), T, Cin,
        Cout, block, rank, _xbar_fmt(xbar_bits, xbar_per_channel), _ptr(r["g_w"]), _ptr(ws),
        _ws_bytes(ws, dev.index), _ptr(r["qg"]),
        _ptr(r["sg"]), _ptr(r["acc"]), _stream(stream)), "hlq_debug_gw_parts")
    return r


def hlq_debug_hq_transform(src, axis: int, stream=None):
    """fp32 Hadamard coefficients of src [rows, cols] along cols (axis 0) or
    rows (axis 1), each the exact sum rounded once to fp32."""
    torch = _torch()
    _need_cuda_contig(src)
    rows, cols = src.shape
    y = torch.empty((rows, cols), dtype=torch.float32, device=src.device)
    _check(lib().hlq_debug_hq_transform(_ptr(src), _dtype_code(src), rows,
                                        cols, axis, _ptr(y), _stream(stream)),
           "hlq_debug_hq_transform")
    return y


def hlq_debug_hla_transform(src, rank: int = 8, stream=None):
    """fp32 HLA coefficients [C, T*rank/16] of src [T, C]."""
    torch = _torch()
    _need_cuda_contig(src)
    T, C = src.shape
    out = torch.empty((C, T // 16 * rank), dtype=torch.float32,
                      device=src.device)
    _check(lib().hlq_debug_hla_transform(_ptr(src), _dtype_code(src), T, C,
                                         rank, _ptr(out), _stream(stream)),
           "hlq_debug_hla_transform")
    return out


def hlq_debug_reference_gemm(a, b, stream=None):
    """int32 a @ b^T of int8 code matrices a [M, K], b [N, K] on CUDA cores."""
    torch = _torch()
    _need_cuda_contig(a, b)
    M, K = a.shape
    N = b.shape[0]
    acc = torch.empty((M, N), dtype=torch.int32, device=a.device)
    _check(lib().hlq_debug_reference_gemm(0, _ptr(a), _ptr(b), M, N, K,
                                          _ptr(acc), _stream(stream)),
           "hlq_debug_reference_gemm")
    return acc


def hlq_debug_wait_timeout(limit_ns: int = 1_000_000, stream=None):
    """Run the bounded-wait failure path once (a wait nothing completes,
    given up after limit_ns): returns the device int32 result (0)."""
    torch = _torch()
    out = torch.full((4,), -1, dtype=torch.int32, device=torch.cuda.current_device())
    _check(lib().hlq_debug_wait_timeout(int(limit_ns), _ptr(out), _stream(stream)),
           "hlq_debug_wait_timeout")
    return out[:1]


def hlq_debug_gemm_plan(T: int, Cin: int, Cout: int, rank: int = 8, sms: int = 152):
    """The GEMM plans of a layer on a GPU with `sms` SMs (host only): dict of
    gx (bn, splits), gw (bn, splits) and in_sequence."""
    vals = [ctypes.c_int(0) for _ in range(7)]
    _check(lib().hlq_debug_gemm_plan(T, Cin, Cout, rank, sms,
                                     *[ctypes.byref(v) for v in vals]),
           "hlq_debug_gemm_plan")
    g = [v.value for v in vals]
    return {"gx": (g[0], g[1]), "gw": (g[2], g[3]), "in_sequence": bool(g[4]),
            "gx_pair": bool(g[5]), "gw_pair": bool(g[6])}


def hlq_debug_tc_gemm(kind, a, b, bn=0, splits=0, pair=-1, stream=None):
    """int32 a @ b^T on the tensor cores with an explicit plan.  kind 0: a, b
    are uint8 E4M3 codes [M, K] / [N, K]; kind 1: fp16 codes; kind 2: a fp16,
    b int8 codes (widened in the GEMM); kind 3: a and b int8.  pair: 1 = CTA
    pairs over 256-row tiles, 0 = one CTA per 128-row tile, -1 = the
    library's choice."""
    torch = _torch()
    _need_cuda_contig(a, b)
    M, K = a.shape
    N = b.shape[0]
    acc = torch.empty((M, N), dtype=torch.int32, device=a.device)
    nws = int(lib().hlq_debug_tc_gemm_ws_bytes(M, N))
    ws = torch.empty(max(nws, 256), dtype=torch.uint8, device=a.device)
    _check(lib().hlq_debug_tc_gemm(kind, _ptr(a), K, _ptr(b), K, M, N, K, bn,
                                   splits, pair, _ptr(acc), _ptr(ws),
                                   _ws_bytes(ws, a.device.index),
                                   _stream(stream)), "hlq_debug_tc_gemm")
    return acc


GW_AUTO, GW_WIDEN, GW_INT8_X, GW_INT8_BOTH = 0, 1, 2, 3


def hlq_set_gw_operands(mode: int):
    """How the g_w GEMMs take their int8 operands, for the whole process:
    GW_WIDEN (x-bar widened to fp16 by its own kernel), GW_INT8_X (the GEMM
    widens x-bar tiles in shared memory), GW_INT8_BOTH (the HLA codes of g_y
    stay int8 too), GW_AUTO (the library's default).  Results are identical
    in every mode."""
    _check(lib().hlq_set_gw_operands(int(mode)), "hlq_set_gw_operands")


def hlq_get_gw_operands() -> int:
    return int(lib().hlq_get_gw_operands())


def hlq_debug_serialize_branches(on: bool):
    """Run the branches of hlq_linear_backward / hlq_layer_step on the
    caller's stream one after the other (same kernels, for per-kernel
    timing), or forked again (on=False)."""
    _check(lib().hlq_debug_serialize_branches(1 if on else 0),
           "hlq_debug_serialize_branches")


def hlq_trace_begin(capacity: int = 4096):
    """Start recording per-launch device times of libhlq's kernels."""
    _check(lib().hlq_trace_begin(capacity), "hlq_trace_begin")


_trace_n = 0


def hlq_trace_end(keep: bool = False):
    """Stop tracing; return [(kernel name, ms), ...] in launch order.  With
    keep=True return the number of traced launches and keep the events
    alive (for graph replays: hlq_trace_read() after each replay, then
    hlq_trace_free())."""
    global _trace_n
    L = lib()
    n = ctypes.c_int(0)
    _check(L.hlq_trace_end(ctypes.byref(n)), "hlq_trace_end")
    _trace_n = n.value
    if keep:
        return _trace_n
    out = hlq_trace_read()
    L.hlq_trace_free()
    return out


def hlq_trace_read():
    """Per-launch (name, ms) of the last recording of the traced launches."""
    L = lib()
    out = []
    for i in range(_trace_n):
        name = ctypes.c_char_p()
        ms = ctypes.c_float()
        _check(L.hlq_trace_get(i, ctypes.byref(name), ctypes.byref(ms)),
               "hlq_trace_get")
        out.append((name.value.decode(), float(ms.value)))
    return out


def hlq_trace_free():
    lib().hlq_trace_free()


def hlq_read_device_status(clear: bool = False, stream=None) -> int:
    flags = ctypes.c_uint32(0)
    _check(lib().hlq_read_device_status(ctypes.byref(flags), 1 if clear else 0,
                                        _stream(stream)),
           "hlq_read_device_status")
    return int(flags.value)

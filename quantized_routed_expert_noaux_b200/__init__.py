"""Python binding of libcoli_moe.so: the routed-expert MoE layer on B200 (sm_100a).

Argument marshalling only.  Every function has the name of the C entry point it calls
(include/coli_moe.h), takes torch CUDA tensors (or None for a NULL pointer), passes their
device pointers and the current torch CUDA stream, and raises ColiError on a non-OK status.
Every step of the layer runs in the library's CUDA kernels; there is no CPU path.  Importing
this package raises ImportError when the library has not been built.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Optional

__all__ = [
    "ColiError", "MoEConfig", "MoEWeights", "lib", "LIB_PATH",
    "coli_moe_status_str", "coli_moe_last_cuda_error", "coli_moe_record_bytes", "coli_moe_check_config",
    "coli_moe_workspace_size", "coli_moe_clear_error", "coli_moe_error_word",
    "coli_moe_gate", "coli_moe_route", "coli_moe_group", "coli_moe_ffn", "coli_moe_layer",
    "coli_moe_layer_noalloc", "coli_moe_noalloc_error_word", "STATIC_SCRATCH_BYTES", "coli_moe_layer_kernels", "coli_moe_residual",
    "coli_moe_debug_set_wait",
    "coli_moe_set_dispatch_threshold",
    "coli_moe_dispatch_threshold",
    "config_for", "weights_for",
    "MoERouter", "coli_moe_check_router", "coli_moe_route_scores",
    "FP4Rows", "FP4Mats", "coli_moe_fp4_scale_pitch", "coli_moe_fp4_scale_bytes", "coli_moe_fp4_quantize",
    "coli_moe_fp4_dequantize", "coli_moe_fp4_product", "coli_moe_fp4_pack_record", "fp4_rows_for", "fp4_mats_for",
    "coli_moe_sort_rows", "coli_moe_combine", "coli_moe_combine_grad",
    "I8Rows", "I8Mats", "coli_moe_i8_quantize", "coli_moe_i8_product", "i8_rows_for", "i8_mats_for",
    "COLI_W_NVFP4", "COLI_W_MXFP4", "COLI_SCORE_SIGMOID", "COLI_SCORE_SOFTMAX", "COLI_GROUP_TOP2", "COLI_GROUP_MAX",
    "COLI_FP4_MX", "COLI_FP4_NV", "COLI_FP4_ROWS", "COLI_FP4_TILES",
    "COLI_W_INT2", "COLI_W_INT4", "COLI_W_INT8", "COLI_ACT_F32", "COLI_ACT_BF16",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcoli_moe.so")

COLI_W_INT2, COLI_W_INT4, COLI_W_INT8 = 2, 4, 8
COLI_W_NVFP4, COLI_W_MXFP4 = 20, 36
COLI_ACT_F32, COLI_ACT_BF16 = 0, 1
COLI_SCORE_SIGMOID, COLI_SCORE_SOFTMAX = 0, 1
COLI_GROUP_TOP2, COLI_GROUP_MAX = 0, 1
COLI_FP4_MX, COLI_FP4_NV = 0, 1
COLI_FP4_ROWS, COLI_FP4_TILES = 0, 1
DEVERR_EXPERT_ID, DEVERR_GROUPING, DEVERR_TIMEOUT = 0x1, 0x2, 0x4

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python quantized_routed_expert_noaux_b200/build.py` "
        "(there is no CPU fallback for this layer)")


class MoEConfig(C.Structure):
    _fields_ = [
        ("hidden", C.c_int), ("inter", C.c_int), ("n_experts", C.c_int), ("top_k", C.c_int),
        ("n_group", C.c_int), ("topk_group", C.c_int), ("n_shared", C.c_int),
        ("shared_inter", C.c_int), ("routed_scaling", C.c_double), ("wfmt", C.c_int),
        ("act", C.c_int), ("group_size", C.c_int),
    ]


class MoEWeights(C.Structure):
    _fields_ = [
        ("router_w", C.c_void_p), ("router_bias", C.c_void_p), ("experts", C.c_void_p),
        ("expert_stride", C.c_size_t), ("shared", C.c_void_p),
    ]


class MoERouter(C.Structure):
    """coli_moe_router: the description of a router from scores (coli_moe_route_scores)."""
    _fields_ = [
        ("n_experts", C.c_int), ("top_k", C.c_int), ("n_group", C.c_int), ("topk_group", C.c_int),
        ("score", C.c_int), ("group_score", C.c_int), ("renorm", C.c_int), ("logits", C.c_int),
        ("scaling", C.c_double),
    ]


class FP4Rows(C.Structure):
    device = None  # of the tensors that fp4_rows_for took
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("row_scale", C.c_void_p), ("rows", C.c_int)]


class FP4Mats(C.Structure):
    device = None
    _fields_ = [
        ("codes", C.c_void_p), ("scales", C.c_void_p), ("row_scale", C.c_void_p), ("count", C.c_int), ("n", C.c_int),
        ("codes_stride", C.c_size_t), ("scales_stride", C.c_size_t), ("row_scale_stride", C.c_size_t),
    ]


class I8Rows(C.Structure):
    device = None  # of the tensors that i8_rows_for took
    _fields_ = [("codes", C.c_void_p), ("scale", C.c_void_p), ("rows", C.c_int), ("ld", C.c_size_t)]


class I8Mats(C.Structure):
    device = None
    _fields_ = [
        ("codes", C.c_void_p), ("scale", C.c_void_p), ("count", C.c_int), ("n", C.c_int),
        ("ld", C.c_size_t), ("codes_stride", C.c_size_t), ("scale_stride", C.c_size_t),
    ]


class ColiError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        extra = ""
        if status == 5:
            extra = " [" + lib.coli_moe_last_cuda_error().decode() + "]"
        super().__init__(f"{fn}: {coli_moe_status_str(status)} (status {status}){extra}")


def _load():
    L = C.CDLL(LIB_PATH)
    P, I, S = C.c_void_p, C.c_int, C.c_size_t
    cfgp, wp = C.POINTER(MoEConfig), C.POINTER(MoEWeights)
    L.coli_moe_status_str.argtypes = [I]
    L.coli_moe_status_str.restype = C.c_char_p
    L.coli_moe_last_cuda_error.argtypes = []
    L.coli_moe_last_cuda_error.restype = C.c_char_p
    L.coli_moe_record_bytes.argtypes = [I, I, I, I, C.POINTER(S)]
    L.coli_moe_check_config.argtypes = [cfgp]
    L.coli_moe_workspace_size.argtypes = [cfgp, I, C.POINTER(S)]
    L.coli_moe_clear_error.argtypes = [P, P]
    L.coli_moe_error_word.argtypes = [P, P, C.POINTER(I)]
    L.coli_moe_gate.argtypes = [cfgp, P, P, I, P, P]
    L.coli_moe_route.argtypes = [cfgp, P, P, I, P, P, P]
    L.coli_moe_group.argtypes = [cfgp, P, I, P, P, P, P, P, P, S, P]
    L.coli_moe_ffn.argtypes = [cfgp, wp, P, I, P, P, P, P, P, P, P, S, P]
    L.coli_moe_layer.argtypes = [cfgp, wp, P, I, P, P, P, P, S, P]
    L.coli_moe_layer_noalloc.argtypes = [cfgp, wp, P, I, P, P, P, P]
    L.coli_moe_noalloc_error_word.argtypes = [P, C.POINTER(I)]
    L.coli_moe_layer_kernels.argtypes = [cfgp, I, C.POINTER(I)]
    L.coli_moe_residual.argtypes = [cfgp, P, P, I, P, P]
    L.coli_moe_debug_set_wait.argtypes = [C.c_longlong, I]
    L.coli_moe_set_dispatch_threshold.argtypes = [I]
    L.coli_moe_dispatch_threshold.argtypes = []
    L.coli_moe_dispatch_threshold.restype = I
    L.coli_moe_check_router.argtypes = [C.POINTER(MoERouter)]
    L.coli_moe_route_scores.argtypes = [C.POINTER(MoERouter), P, S, P, I, P, P, P]
    L.coli_moe_fp4_scale_pitch.argtypes = [I, I, C.POINTER(S)]
    L.coli_moe_fp4_scale_bytes.argtypes = [I, I, I, I, C.POINTER(S)]
    L.coli_moe_fp4_quantize.argtypes = [I, I, I, P, I, S, P, I, I, I, P, P, P, P, P]
    L.coli_moe_fp4_dequantize.argtypes = [I, I, P, P, P, I, I, I, P, S, P]
    L.coli_moe_fp4_pack_record.argtypes = [cfgp, I, P, P, P, P, P, P]
    L.coli_moe_fp4_product.argtypes = [I, C.POINTER(FP4Rows), C.POINTER(FP4Mats), I, P, I, P, S, P, P]
    L.coli_moe_sort_rows.argtypes = [I, I, I, P, I, I, S, P, P, P, P, P, S, P, P]
    L.coli_moe_combine.argtypes = [I, P, I, S, P, P, I, I, I, I, P, S, P, S, P, P]
    L.coli_moe_combine_grad.argtypes = [I, P, I, S, P, P, I, I, I, I, P, S, P, S, P, P, P]
    L.coli_moe_i8_quantize.argtypes = [I, I, P, I, S, I, P, I, I, P, S, P, P, P]
    L.coli_moe_i8_product.argtypes = [C.POINTER(I8Rows), C.POINTER(I8Mats), I, P, I, P, S, P, P]
    L.coli_moe_layer_kernels.restype = I
    L.coli_moe_layer_noalloc.restype = I
    for name in ("coli_moe_record_bytes", "coli_moe_check_config", "coli_moe_workspace_size",
                 "coli_moe_clear_error", "coli_moe_error_word", "coli_moe_gate",
                 "coli_moe_route", "coli_moe_group", "coli_moe_ffn", "coli_moe_layer",
                 "coli_moe_residual", "coli_moe_debug_set_wait", "coli_moe_set_dispatch_threshold",
                 "coli_moe_noalloc_error_word", "coli_moe_check_router", "coli_moe_route_scores",
                 "coli_moe_fp4_scale_pitch", "coli_moe_fp4_scale_bytes", "coli_moe_fp4_quantize",
                 "coli_moe_fp4_dequantize", "coli_moe_fp4_product", "coli_moe_fp4_pack_record",
                 "coli_moe_sort_rows", "coli_moe_combine", "coli_moe_combine_grad", "coli_moe_i8_quantize",
                 "coli_moe_i8_product"):
        getattr(L, name).restype = I
    return L


lib = _load()


def _p(t) -> Optional[int]:
    return t if t is None or t.__class__ is int else t.data_ptr()


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _stream(stream) -> Optional[int]:
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return _current_stream()


# torch's own functions for the current device and the handle of its current stream.  The handle alone:
# building torch's Stream object takes longer (3.3 us against 0.1) than launching a small kernel.
_torch_device = _torch_stream = None


def _current_stream() -> int:
    global _torch_device, _torch_stream
    if _torch_device is None:
        import torch
        if not torch.cuda.is_initialized() or not hasattr(torch._C, "_cuda_getCurrentRawStream"):
            return torch.cuda.current_stream().cuda_stream
        _torch_device, _torch_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    return _torch_stream(_torch_device())


def _stream_at(fn: str, stream, at: int, together: bool) -> Optional[int]:
    """_stream for a call whose tensors lie on CUDA device `at`, all of them if `together`: the current one it must be."""
    if not together or at < 0:  # (-1: not a CUDA tensor)
        raise ColiError(fn, 1)
    if _torch_device is None:
        _current_stream()
    if _torch_device is not None and at != _torch_device():
        raise ColiError(fn, 1)
    if stream is not None:
        return stream if stream.__class__ is int else stream.cuda_stream
    return _torch_stream(at) if _torch_device is not None else _current_stream()


def _pointers(fn: str, stream, *tensors):
    """The same for tensors, device pointers and None in any mixture: their pointers and the stream."""
    devices = [t.get_device() for t in tensors if t is not None and t.__class__ is not int]
    st = _stream_at(fn, stream, devices[0], devices.count(devices[0]) == len(devices)) if devices else _stream(stream)
    return *map(_p, tensors), st


def _product_pointers(fn: str, stream, a, w, *tensors):
    """_pointers for a product, whose operands are structures that may know their device: theirs and the tensors' is one."""
    devices = {getattr(m, "device", None) for m in (a, w)} - {None}
    devices |= {t.get_device() for t in tensors if t is not None and t.__class__ is not int}
    st = _stream_at(fn, stream, min(devices), len(devices) == 1) if devices else _stream(stream)
    return *map(_p, tensors), st


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise ColiError(fn, status)


def coli_moe_status_str(status: int) -> str:
    return lib.coli_moe_status_str(status).decode()


def coli_moe_last_cuda_error() -> str:
    return lib.coli_moe_last_cuda_error().decode()


def coli_moe_record_bytes(hidden: int, inter: int, wfmt: int, group_size: int = 0) -> int:
    n = C.c_size_t()
    _check("coli_moe_record_bytes", lib.coli_moe_record_bytes(hidden, inter, wfmt, group_size, C.byref(n)))
    return n.value


def coli_moe_check_config(cfg: MoEConfig) -> None:
    _check("coli_moe_check_config", lib.coli_moe_check_config(C.byref(cfg)))


def coli_moe_workspace_size(cfg: MoEConfig, max_tokens: int) -> int:
    n = C.c_size_t()
    _check("coli_moe_workspace_size",
           lib.coli_moe_workspace_size(C.byref(cfg), max_tokens, C.byref(n)))
    return n.value


def coli_moe_clear_error(ws, stream=None) -> None:
    _check("coli_moe_clear_error", lib.coli_moe_clear_error(_p(ws), _stream(stream)))


def coli_moe_error_word(ws, stream=None) -> int:
    v = C.c_int()
    _check("coli_moe_error_word", lib.coli_moe_error_word(_p(ws), _stream(stream), C.byref(v)))
    return v.value


def coli_moe_layer_kernels(cfg, T) -> int:
    n = C.c_int()
    _check("coli_moe_layer_kernels", lib.coli_moe_layer_kernels(C.byref(cfg), T, C.byref(n)))
    return n.value


def coli_moe_gate(cfg, router_w, x, T, logits, stream=None) -> None:
    _check("coli_moe_gate", lib.coli_moe_gate(C.byref(cfg), _p(router_w), _p(x), T, _p(logits),
                                              _stream(stream)))


def coli_moe_route(cfg, logits, bias, T, topk_ids, topk_w, stream=None) -> None:
    _check("coli_moe_route", lib.coli_moe_route(C.byref(cfg), _p(logits), _p(bias), T,
                                                _p(topk_ids), _p(topk_w), _stream(stream)))


def coli_moe_group(cfg, topk_ids, T, counts, offsets, perm, unique_ids, n_unique, ws,
                   stream=None) -> None:
    _check("coli_moe_group", lib.coli_moe_group(
        C.byref(cfg), _p(topk_ids), T, _p(counts), _p(offsets), _p(perm), _p(unique_ids),
        _p(n_unique), _p(ws), _nbytes(ws), _stream(stream)))


def coli_moe_ffn(cfg, weights: MoEWeights, x, T, topk_w, offsets, perm, unique_ids, n_unique,
                 out, ws, stream=None) -> None:
    _check("coli_moe_ffn", lib.coli_moe_ffn(
        C.byref(cfg), C.byref(weights), _p(x), T, _p(topk_w), _p(offsets), _p(perm),
        _p(unique_ids), _p(n_unique), _p(out), _p(ws), _nbytes(ws), _stream(stream)))


def coli_moe_layer(cfg, weights: MoEWeights, x, T, out, topk_ids_out, topk_w_out, ws,
                   stream=None) -> None:
    _check("coli_moe_layer", lib.coli_moe_layer(
        C.byref(cfg), C.byref(weights), _p(x), T, _p(out), _p(topk_ids_out), _p(topk_w_out),
        _p(ws), _nbytes(ws), _stream(stream)))


def coli_moe_residual(cfg, x, out, T, x_next, stream=None) -> None:
    """x_next = x + out between chained layers (float32 sum; bf16 activations rounded to bf16)."""
    _check("coli_moe_residual", lib.coli_moe_residual(
        C.byref(cfg), _p(x), _p(out), T, _p(x_next), _stream(stream)))


# Size of the static scratch array behind coli_moe_layer_noalloc (COLI_MOE_STATIC_SCRATCH_BYTES).
STATIC_SCRATCH_BYTES = 8 << 20


def coli_moe_layer_noalloc(cfg, weights: MoEWeights, x, T, out, topk_ids_out=None,
                           topk_w_out=None, stream=None) -> None:
    """The whole layer for callers that cannot allocate device memory (a plugin whose GPU memory
    pool is fixed at start-up, a real-time loop that cannot afford cudaMalloc's synchronisation):
    no workspace argument; the library's static per-GPU scratch array is used instead.  Calls on
    one device share that array, so calls that overlap on the GPU must be ordered."""
    _check("coli_moe_layer_noalloc", lib.coli_moe_layer_noalloc(
        C.byref(cfg), C.byref(weights), _p(x), T, _p(out), _p(topk_ids_out), _p(topk_w_out),
        _stream(stream)))


def coli_moe_noalloc_error_word(stream=None) -> int:
    """Device error word of the static scratch array behind coli_moe_layer_noalloc (synchronises
    the stream): 0 when the last no-allocation call on this device ran clean."""
    v = C.c_int()
    _check("coli_moe_noalloc_error_word", lib.coli_moe_noalloc_error_word(_stream(stream), C.byref(v)))
    return v.value


def coli_moe_debug_set_wait(wait_cycles: int, unreachable: bool) -> None:
    """Testing aid: the fused decode kernel's wait bound (cycles, 0 = default) and whether its
    grid-barrier targets are out of reach (every wait then runs out and reports a timeout)."""
    _check("coli_moe_debug_set_wait", lib.coli_moe_debug_set_wait(wait_cycles, int(bool(unreachable))))


def coli_moe_set_dispatch_threshold(max_tokens: int) -> None:
    """a5' per-expert dispatch on the tensor-core path: work experts with at most max_tokens
    routed tokens take the CUDA-core GEMV kernels, the rest the grouped GEMM (0: all GEMM)."""
    _check("coli_moe_set_dispatch_threshold", lib.coli_moe_set_dispatch_threshold(int(max_tokens)))


def coli_moe_dispatch_threshold() -> int:
    """The current per-expert dispatch threshold."""
    return int(lib.coli_moe_dispatch_threshold())


def config_for(wl) -> MoEConfig:
    """MoEConfig with the shape fields of a workload description (any object with the
    attributes hidden, inter, n_experts, top_k, n_group, topk_group, n_shared, shared_inter,
    routed_scaling, fmt and act = "f32" | "bf16")."""
    return MoEConfig(wl.hidden, wl.inter, wl.n_experts, wl.top_k, wl.n_group, wl.topk_group,
                     wl.n_shared, wl.shared_inter, float(wl.routed_scaling), wl.fmt,
                     COLI_ACT_F32 if wl.act == "f32" else COLI_ACT_BF16, getattr(wl, "group", 0))


def weights_for(router_w, router_bias, experts, shared=None) -> MoEWeights:
    """MoEWeights over device tensors: experts is [E, stride] uint8, shared [stride_s] uint8."""
    return MoEWeights(_p(router_w), _p(router_bias), _p(experts), experts.stride(0),
                      _p(shared))


def coli_moe_check_router(router: MoERouter) -> None:
    _check("coli_moe_check_router", lib.coli_moe_check_router(C.byref(router)))


_c_route_scores, _c_fp4_quantize = lib.coli_moe_route_scores, lib.coli_moe_fp4_quantize
_c_fp4_dequantize, _c_fp4_product = lib.coli_moe_fp4_dequantize, lib.coli_moe_fp4_product

# The calls below may run every few microseconds (one decoded token through a router or a linear layer), so
# they pass structures and pointers to ctypes without helpers in between.  All tensors of a call must live on the
# current device: one that does not would be a bad address to the kernel.

def coli_moe_route_scores(router: MoERouter, logits, ld, bias, T, topk_ids, topk_w, stream=None) -> None:
    """Softmax or sigmoid routing of T tokens: row t of the logits at element t * ld (0: n_experts),
    bias [E] float32 or None."""
    try:
        at = logits.get_device()
        together = at == topk_ids.get_device() == topk_w.get_device() and (bias is None or at == bias.get_device())
        st = (_torch_stream(at) if together and stream is None and _torch_device is not None and at == _torch_device()
              else _stream_at("coli_moe_route_scores", stream, at, together))
        status = _c_route_scores(router, logits.data_ptr(), ld, None if bias is None else bias.data_ptr(), T, topk_ids.data_ptr(),
                                           topk_w.data_ptr(), st)
    except AttributeError:  # device pointers among them
        logits, bias, topk_ids, topk_w, st = _pointers("coli_moe_route_scores", stream, logits, bias, topk_ids, topk_w)
        status = _c_route_scores(router, logits, ld, bias, T, topk_ids, topk_w, st)
    if status:
        raise ColiError("coli_moe_route_scores", status)


def coli_moe_fp4_scale_pitch(fmt: int, k: int) -> int:
    n = C.c_size_t()
    _check("coli_moe_fp4_scale_pitch", lib.coli_moe_fp4_scale_pitch(fmt, k, C.byref(n)))
    return n.value


def coli_moe_fp4_scale_bytes(fmt: int, layout: int, rows: int, k: int) -> int:
    n = C.c_size_t()
    _check("coli_moe_fp4_scale_bytes", lib.coli_moe_fp4_scale_bytes(fmt, layout, rows, k, C.byref(n)))
    return n.value


def coli_moe_fp4_quantize(fmt, layout, act, x, src_rows, ldx, row_index, row_div, rows, k, codes, scales, row_scale, ws,
                          stream=None) -> None:
    """Rows of x (row i at element i * ldx) to 4-bit codes, block scales and row scales; row r of the
    result is source row r, or row_index[r] // row_div."""
    try:
        at = x.get_device()
        together = (at == codes.get_device() == scales.get_device() == row_scale.get_device() == ws.get_device() and
                    (row_index is None or at == row_index.get_device()))
        st = (_torch_stream(at) if together and stream is None and _torch_device is not None and at == _torch_device()
              else _stream_at("coli_moe_fp4_quantize", stream, at, together))
        status = _c_fp4_quantize(fmt, layout, act, x.data_ptr(), src_rows, ldx, None if row_index is None else row_index.data_ptr(), row_div,
                                           rows, k, codes.data_ptr(), scales.data_ptr(), row_scale.data_ptr(), ws.data_ptr(), st)
    except AttributeError:
        x, row_index, codes, scales, row_scale, ws, st = _pointers("coli_moe_fp4_quantize", stream, x, row_index, codes, scales, row_scale, ws)
        status = _c_fp4_quantize(fmt, layout, act, x, src_rows, ldx, row_index, row_div, rows, k, codes, scales, row_scale, ws, st)
    if status:
        raise ColiError("coli_moe_fp4_quantize", status)


def coli_moe_fp4_dequantize(fmt, layout, codes, scales, row_scale, rows, k, act, out, ldo, stream=None) -> None:
    """The values that codes, block scales and row scales stand for, rounded to act; row r at out + r * ldo."""
    try:
        at = out.get_device()
        together = at == codes.get_device() == scales.get_device() and (row_scale is None or at == row_scale.get_device())
        st = (_torch_stream(at) if together and stream is None and _torch_device is not None and at == _torch_device()
              else _stream_at("coli_moe_fp4_dequantize", stream, at, together))
        status = _c_fp4_dequantize(fmt, layout, codes.data_ptr(), scales.data_ptr(), None if row_scale is None else row_scale.data_ptr(), rows, k,
                                             act, out.data_ptr(), ldo, st)
    except AttributeError:
        codes, scales, row_scale, out, st = _pointers("coli_moe_fp4_dequantize", stream, codes, scales, row_scale, out)
        status = _c_fp4_dequantize(fmt, layout, codes, scales, row_scale, rows, k, act, out, ldo, st)
    if status:
        raise ColiError("coli_moe_fp4_dequantize", status)


def coli_moe_fp4_product(fmt, a: FP4Rows, w: FP4Mats, k, offsets, out_type, out, ldo, ws, stream=None) -> None:
    """out row i = a's row i times the matrix of its group (offsets [count + 1] int32; None: one matrix)."""
    try:
        at = out.get_device()
        together = (at == ws.get_device() and (offsets is None or at == offsets.get_device()) and
                    (a.device is None or at == a.device) and (w.device is None or at == w.device))
        st = (_torch_stream(at) if together and stream is None and _torch_device is not None and at == _torch_device()
              else _stream_at("coli_moe_fp4_product", stream, at, together))
        status = _c_fp4_product(fmt, a, w, k, None if offsets is None else offsets.data_ptr(), out_type, out.data_ptr(), ldo, ws.data_ptr(), st)
    except AttributeError:
        offsets, out, ws, st = _product_pointers("coli_moe_fp4_product", stream, a, w, offsets, out, ws)
        status = _c_fp4_product(fmt, a, w, k, offsets, out_type, out, ldo, ws, st)
    if status:
        raise ColiError("coli_moe_fp4_product", status)


def coli_moe_fp4_pack_record(cfg: MoEConfig, act, wg, wu, wd, record, ws, stream=None) -> None:
    """One expert's gate, up [I, H] and down [H, I] matrices into a record of cfg's 4-bit container."""
    wg, wu, wd, record, ws, st = _pointers("coli_moe_fp4_pack_record", stream, wg, wu, wd, record, ws)
    _check("coli_moe_fp4_pack_record", lib.coli_moe_fp4_pack_record(C.byref(cfg), act, wg, wu, wd, record, ws, st))


_int8 = _float32 = None  # torch's types, once a tensor has come


def _types() -> None:
    global _int8, _float32
    import torch
    _int8, _float32 = torch.int8, torch.float32


# The helpers refuse arrays that the kernels would read behind their end, or as what they are not: a few comparisons.  Block scales: at least
# 8 bytes of a row per 128 of its codes (MX; NV has twice as many).

def fp4_rows_for(codes, scales, row_scale=None) -> FP4Rows:
    """FP4Rows over device tensors: codes [rows, k/2] uint8, scales [rows, pitch] uint8, row_scale [rows],
    all of them contiguous (the kernels take no strides for them)."""
    at = codes.get_device()
    if row_scale is None:
        row, dense, together = None, codes.is_contiguous() and scales.is_contiguous(), at == scales.get_device()
    else:
        row, dense = row_scale.data_ptr(), codes.is_contiguous() and scales.is_contiguous() and row_scale.is_contiguous()
        together = at == scales.get_device() == row_scale.get_device()
    if _float32 is None:
        _types()
    if codes.dim() != 2:
        raise ColiError("fp4_rows_for", 2)
    rows, half = codes.shape
    if not dense or (row is not None and row_scale.shape != (rows,)) or scales.numel() < rows * 8 * ((half + 127) // 128):
        raise ColiError("fp4_rows_for", 2)
    if not together or at < 0 or not codes.element_size() == scales.element_size() == 1 or (row is not None and row_scale.dtype is not _float32):
        raise ColiError("fp4_rows_for", 1)
    a = FP4Rows(codes.data_ptr(), scales.data_ptr(), row, rows)
    a.device = at
    return a


def fp4_mats_for(codes, scales, row_scale=None) -> FP4Mats:
    """FP4Mats over device tensors: codes [count, n, k/2] uint8, scales [count, bytes] uint8 in tiles,
    row_scale [count, n].  Each matrix of a tensor is contiguous; the matrices may lie further apart."""
    at = codes.get_device()
    if codes.dim() != 3 or (row_scale is not None and row_scale.dim() != 2):
        raise ColiError("fp4_mats_for", 2)
    count, n, half = codes.shape
    c, s = codes.stride(), scales.stride()
    if row_scale is None:
        row, r, together = None, (0, 1), at == scales.get_device()
    else:
        row, r, together = row_scale.data_ptr(), row_scale.stride(), at == scales.get_device() == row_scale.get_device()
    if not (c[2] == 1 and c[1] == half and len(s) == 2 and s[1] == 1 and r[1] == 1):  # (dimensions of one element may have any stride)
        if not all(t is None or t.is_contiguous() or t[0].is_contiguous() for t in (codes, scales, row_scale)):
            raise ColiError("fp4_mats_for", 2)
    if _float32 is None:
        _types()
    if ((row is not None and row_scale.shape != (count, n)) or scales.shape[0] != count or
            scales.numel() < count * ((n + 127) // 128) * 1024 * ((half + 127) // 128)):
        raise ColiError("fp4_mats_for", 2)
    if not together or at < 0 or not codes.element_size() == scales.element_size() == 1 or (row is not None and row_scale.dtype is not _float32):
        raise ColiError("fp4_mats_for", 1)
    w = FP4Mats(codes.data_ptr(), scales.data_ptr(), row, count, n, c[0], s[0], r[0])
    w.device = at
    return w


# ------------------------------------------------------------------ rows to the experts and back, 8-bit products

_c_sort_rows, _c_combine, _c_combine_grad = lib.coli_moe_sort_rows, lib.coli_moe_combine, lib.coli_moe_combine_grad
_c_i8_quantize, _c_i8_product = lib.coli_moe_i8_quantize, lib.coli_moe_i8_product


def _quick(fn: str, stream, at: int, together: bool) -> Optional[int]:
    """The stream of a call whose tensors lie on device `at`: the usual case without helpers in between."""
    if together and stream is None and _torch_device is not None and at == _torch_device():
        return _torch_stream(at)
    return _stream_at(fn, stream, at, together)


def coli_moe_sort_rows(n_experts, top_k, act, x, T, hidden, ldx, topk_ids, offsets, perm, place, rows, ldr, ws, stream=None) -> None:
    """Slots sorted by expert: offsets [n_experts + 1], perm and place [T * top_k], and the slots' rows of x
    (x and rows None: the sort alone).  An id of -1 leaves its slot out."""
    try:
        at = ws.get_device()
        together = (at == topk_ids.get_device() == offsets.get_device() == perm.get_device() == place.get_device() and
                    (x is None or at == x.get_device()) and (rows is None or at == rows.get_device()))
        st = _quick("coli_moe_sort_rows", stream, at, together)
        status = _c_sort_rows(n_experts, top_k, act, None if x is None else x.data_ptr(), T, hidden, ldx, topk_ids.data_ptr(), offsets.data_ptr(),
                              perm.data_ptr(), place.data_ptr(), None if rows is None else rows.data_ptr(), ldr, ws.data_ptr(), st)
    except AttributeError:  # device pointers or None among them
        x, topk_ids, offsets, perm, place, rows, ws, st = _pointers("coli_moe_sort_rows", stream, x, topk_ids, offsets, perm, place, rows, ws)
        status = _c_sort_rows(n_experts, top_k, act, x, T, hidden, ldx, topk_ids, offsets, perm, place, rows, ldr, ws, st)
    if status:
        raise ColiError("coli_moe_sort_rows", status)


def coli_moe_combine(act, y, rows, ldy, place, topk_w, T, top_k, hidden, out_type, add, ld_add, out, ldo, ws, stream=None) -> None:
    """out[t] = add[t] + sum_k topk_w[t, k] * y[place[t, k]] (topk_w None: 1; add None: 0)."""
    try:
        at = out.get_device()
        together = (at == y.get_device() == place.get_device() == ws.get_device() and
                    (topk_w is None or at == topk_w.get_device()) and (add is None or at == add.get_device()))
        st = _quick("coli_moe_combine", stream, at, together)
        status = _c_combine(act, y.data_ptr(), rows, ldy, place.data_ptr(), None if topk_w is None else topk_w.data_ptr(), T, top_k, hidden, out_type,
                            None if add is None else add.data_ptr(), ld_add, out.data_ptr(), ldo, ws.data_ptr(), st)
    except AttributeError:
        y, place, topk_w, add, out, ws, st = _pointers("coli_moe_combine", stream, y, place, topk_w, add, out, ws)
        status = _c_combine(act, y, rows, ldy, place, topk_w, T, top_k, hidden, out_type, add, ld_add, out, ldo, ws, st)
    if status:
        raise ColiError("coli_moe_combine", status)


def coli_moe_combine_grad(act, y, rows, ldy, place, topk_w, T, top_k, hidden, out_type, dout, ld_dout, dy, ld_dy, dw, ws,
                          stream=None) -> None:
    """The gradient of coli_moe_combine: dy rows [place] and dw [T, top_k], either may be None."""
    try:
        at = dout.get_device()
        together = (at == place.get_device() == ws.get_device() and (y is None or at == y.get_device()) and
                    (topk_w is None or at == topk_w.get_device()) and (dy is None or at == dy.get_device()) and (dw is None or at == dw.get_device()))
        st = _quick("coli_moe_combine_grad", stream, at, together)
        status = _c_combine_grad(act, None if y is None else y.data_ptr(), rows, ldy, place.data_ptr(), None if topk_w is None else topk_w.data_ptr(), T,
                                 top_k, hidden, out_type, dout.data_ptr(), ld_dout, None if dy is None else dy.data_ptr(), ld_dy,
                                 None if dw is None else dw.data_ptr(), ws.data_ptr(), st)
    except AttributeError:
        y, place, topk_w, dout, dy, dw, ws, st = _pointers("coli_moe_combine_grad", stream, y, place, topk_w, dout, dy, dw, ws)
        status = _c_combine_grad(act, y, rows, ldy, place, topk_w, T, top_k, hidden, out_type, dout, ld_dout, dy, ld_dy, dw, ws, st)
    if status:
        raise ColiError("coli_moe_combine_grad", status)


def coli_moe_i8_quantize(act, swiglu, x, src_rows, ldx, k, place, copies, rows, codes, ldc, scale, ws, stream=None) -> None:
    """Rows of x (row i at element i * ldx), or SiLU(gate) * up of rows of k gate and k up values, to 8-bit codes with a
    scale each; row i to the rows place[i * copies + c] of the result, or to row i."""
    try:
        at = x.get_device()
        together = at == codes.get_device() == scale.get_device() == ws.get_device() and (place is None or at == place.get_device())
        st = _quick("coli_moe_i8_quantize", stream, at, together)
        status = _c_i8_quantize(act, swiglu, x.data_ptr(), src_rows, ldx, k, None if place is None else place.data_ptr(), copies, rows,
                                codes.data_ptr(), ldc, scale.data_ptr(), ws.data_ptr(), st)
    except AttributeError:
        x, place, codes, scale, ws, st = _pointers("coli_moe_i8_quantize", stream, x, place, codes, scale, ws)
        status = _c_i8_quantize(act, swiglu, x, src_rows, ldx, k, place, copies, rows, codes, ldc, scale, ws, st)
    if status:
        raise ColiError("coli_moe_i8_quantize", status)


def coli_moe_i8_product(a: I8Rows, w: I8Mats, k, offsets, out_type, out, ldo, ws, stream=None) -> None:
    """out row i = a's row i times the matrix of its group (offsets [count + 1] int32; None: one matrix)."""
    try:
        at = out.get_device()
        together = (at == ws.get_device() and (offsets is None or at == offsets.get_device()) and
                    (a.device is None or at == a.device) and (w.device is None or at == w.device))
        st = _quick("coli_moe_i8_product", stream, at, together)
        status = _c_i8_product(a, w, k, None if offsets is None else offsets.data_ptr(), out_type, out.data_ptr(), ldo, ws.data_ptr(), st)
    except AttributeError:
        offsets, out, ws, st = _product_pointers("coli_moe_i8_product", stream, a, w, offsets, out, ws)
        status = _c_i8_product(a, w, k, offsets, out_type, out, ldo, ws, st)
    if status:
        raise ColiError("coli_moe_i8_product", status)


def _fits(codes, dim: int, scale) -> bool:
    """Codes of the type and number of dimensions that the 8-bit kernels take, and scales of theirs."""
    if _int8 is None:
        _types()
    return codes.dim() == dim and codes.dtype is _int8 and (scale is None or scale.dtype is _float32)


def i8_rows_for(codes, scale=None) -> I8Rows:
    """I8Rows over device tensors: codes [rows, >= k] int8, the values of a row side by side, scale [rows] float32, contiguous."""
    if not _fits(codes, 2, scale):
        raise ColiError("i8_rows_for", 2 if codes.dim() != 2 else 1)
    at, r = codes.get_device(), codes.shape[0]
    ld, unit = codes.stride()
    if unit != 1 or not (scale is None or (scale.shape == (r,) and scale.is_contiguous())):
        raise ColiError("i8_rows_for", 2)
    if at < 0 or not (scale is None or scale.get_device() == at):
        raise ColiError("i8_rows_for", 1)
    a = I8Rows(codes.data_ptr(), _p(scale), r, ld)
    a.device = at
    return a


def i8_mats_for(codes, scale=None) -> I8Mats:
    """I8Mats over device tensors: codes [count, n, >= k] int8, the values of a row side by side, scale [count, n] float32 with a
    matrix's scales side by side."""
    if not _fits(codes, 3, scale):
        raise ColiError("i8_mats_for", 2 if codes.dim() != 3 else 1)
    at = codes.get_device()
    count, n, _ = codes.shape
    c = codes.stride()
    if c[2] != 1 or not (scale is None or (scale.shape == (count, n) and scale.stride(1) == 1)):
        raise ColiError("i8_mats_for", 2)
    if at < 0 or not (scale is None or scale.get_device() == at):
        raise ColiError("i8_mats_for", 1)
    w = I8Mats(codes.data_ptr(), _p(scale), count, n, c[1], c[0], 0 if scale is None else scale.stride(0))
    w.device = at
    return w

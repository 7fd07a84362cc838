"""ctypes binding of libqmoe (include/qmoe.h), argument marshalling only.

Each function has the name of the C entry point it calls and takes torch
tensors where the C function takes device pointers; torch supplies device
memory and the current HIP stream and nothing else.  A non-zero status raises
QmoeError.  The library must have been built (python -m
quantized_moe_02_amd.build); there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# QMOE_LIBRARY may name another build of the same library (e.g. a tuning variant)
LIB_PATH = os.environ.get("QMOE_LIBRARY") or os.path.join(_HERE, "libqmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE_TOO_SMALL, MOE_ERR_HIP = range(5)
MOE_WFMT_INT4_G32_F16, MOE_WFMT_NVFP4 = 0, 1
MOE_WFMT_INT4_ROW_F32, MOE_WFMT_INT8_ROW_F32, MOE_WFMT_INT2_ROW_F32 = 2, 3, 4
MOE_OUT_F32, MOE_OUT_BF16 = 0, 1
MOE_OPT_NO_GRID_WAIT, MOE_OPT_GRID_WAIT_NONE, MOE_OPT_INT8_ACTIVATIONS = 1, 2, 4
MOE_FLAG_GRID_WAIT_TIMEOUT = 1
MOE_DT_F32, MOE_DT_BF16, MOE_DT_F16, MOE_DT_MXFP4, MOE_DT_E4M3 = 0, 1, 2, 3, 4
MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = 0, 1
MOE_MAX_TOKENS = 262144
MOE_NOALLOC_WS_BYTES = 32 << 20
WFMT = {"int4": MOE_WFMT_INT4_G32_F16, "nvfp4": MOE_WFMT_NVFP4, "int4_row": MOE_WFMT_INT4_ROW_F32,
        "int8_row": MOE_WFMT_INT8_ROW_F32, "int2_row": MOE_WFMT_INT2_ROW_F32}


class QmoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


class MoeConfig(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("moe_inter", ctypes.c_int32),
                ("n_routed_experts", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("n_shared_experts", ctypes.c_int32), ("shared_inter", ctypes.c_int32),
                ("routed_scaling_factor", ctypes.c_float), ("wfmt", ctypes.c_int32),
                ("options", ctypes.c_uint32), ("expert_top_p", ctypes.c_float)]


class MoeQProj(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("gscale", ctypes.c_void_p)]


class MoeQExperts(ctypes.Structure):
    _fields_ = [("gate", MoeQProj), ("up", MoeQProj), ("down", MoeQProj)]


MOE_TRACE_MAX = 16


class MoeTrace(ctypes.Structure):
    _fields_ = [("events", ctypes.c_void_p * (MOE_TRACE_MAX + 1)), ("n_kernels", ctypes.c_int32),
                ("names", ctypes.c_char_p * MOE_TRACE_MAX)]


class MoeCacheStats(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_uint64), ("hits", ctypes.c_uint64), ("misses", ctypes.c_uint64),
                ("prefetched", ctypes.c_uint64), ("evictions", ctypes.c_uint64),
                ("bytes_loaded", ctypes.c_uint64)]


class MoeMatmulConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("a_rows", ctypes.c_int32),
                ("a_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("lda", ctypes.c_int64), ("ldo", ctypes.c_int64)]


class MoeBalanceConfig(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("n_seq", ctypes.c_int32), ("score", ctypes.c_int32),
                ("logits_dtype", ctypes.c_int32), ("coef", ctypes.c_float)]


class MoeRmsnormConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("residual_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("q_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldh", ctypes.c_int64),
                ("ldy", ctypes.c_int64)]


class MoeRmsnormGradConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("h_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("dy_dtype", ctypes.c_int32),
                ("dx_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("ldh", ctypes.c_int64),
                ("lddy", ctypes.c_int64), ("lddh", ctypes.c_int64), ("lddx", ctypes.c_int64)]


class MoeRowsConfig(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int32), ("cols", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("slots", ctypes.c_int32), ("token_dtype", ctypes.c_int32),
                ("row_dtype", ctypes.c_int32), ("addend_dtype", ctypes.c_int32),
                ("ldt", ctypes.c_int64), ("ldr", ctypes.c_int64), ("lda", ctypes.c_int64)]


class MoeSwigluConfig(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("gu_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("ldg", ctypes.c_int64), ("ldo", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqmoe.so (once).  Raises if it has not been built."""
    global _lib, _several
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m quantized_moe_02_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        cfgp = ctypes.POINTER(MoeConfig)
        exp = ctypes.POINTER(MoeQExperts)
        i64 = ctypes.c_int64
        mmp, balp = ctypes.POINTER(MoeMatmulConfig), ctypes.POINTER(MoeBalanceConfig)
        sig = {
            "moe_workspace_size": [cfgp, i32, ctypes.POINTER(sz)],
            "moe_route": [cfgp, i32, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_permute": [cfgp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_expert_ffn_q4": [cfgp, i32, vp, exp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_combine": [cfgp, i32, vp, vp, vp, vp, vp, i32, vp],
            "moe_layer": [cfgp, i32, vp, vp, vp, exp, exp, vp, i32, vp, vp, vp, sz, vp],
            "moe_layer_trace": [cfgp, i32, vp, vp, vp, exp, exp, vp, i32, vp, vp, vp, sz, vp,
                                ctypes.POINTER(MoeTrace)],
            "moe_layer_flags": [vp, ctypes.POINTER(ctypes.c_uint32), vp],
            "moe_layer_noalloc": [cfgp, i32, vp, vp, vp, exp, exp, vp, i32, vp, vp, vp],
            "moe_cache_create": [cfgp, i32, exp, exp, ctypes.POINTER(vp)],
            "moe_cache_destroy": [vp],
            "moe_layer_cached": [vp, i32, vp, vp, vp, exp, vp, i32, vp, vp, vp, sz, vp],
            "moe_cache_prefetch": [vp, ctypes.POINTER(i32), i32, ctypes.POINTER(i32), vp],
            "moe_cache_pin": [vp, ctypes.POINTER(i32), i32, vp],
            "moe_cache_unpin_all": [vp],
            "moe_cache_get_stats": [vp, ctypes.POINTER(MoeCacheStats)],
            "moe_cache_slot_of": [vp, i32, ctypes.POINTER(i32)],
            "moe_mxfp4_quantize": [vp, i32, i64, i64, i64, vp, vp, vp],
            "moe_mxfp4_dequantize": [vp, vp, i64, i64, vp, i32, i64, vp],
            "moe_mxfp4_matmul": [mmp, vp, vp, vp, vp, vp, vp, vp, vp],
            "moe_mxfp4_matmul_dx": [mmp, vp, vp, vp, vp, vp, vp],
            "moe_balance_workspace_size": [balp, ctypes.POINTER(sz)],
            "moe_balance_loss": [balp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_balance_loss_grad": [balp, vp, vp, vp, vp, vp, vp, vp, vp],
            # the row operators' structs come as packed bytes or by reference
            "moe_rmsnorm": [vp, vp, vp, vp, vp, vp, vp, vp, vp],
            "moe_rmsnorm_workspace_size": [i32, i32, ctypes.POINTER(sz)],
            "moe_rmsnorm_grad": [vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_dispatch": [vp, vp, vp, vp, vp, vp, vp],
            "moe_collect": [vp, vp, vp, vp, vp, vp, vp],
            "moe_collect_grad": [vp, vp, vp, vp, vp, vp, vp, vp],
            "moe_swiglu": [vp, vp, vp, vp, vp, vp],
            "moe_swiglu_grad": [vp, vp, vp, vp, vp, vp],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        _several = torch.cuda.device_count() > 1
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise QmoeError(status, where)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_config(geom: dict, wfmt: str, options: int = 0) -> MoeConfig:
    return MoeConfig(geom["hidden"], geom["moe_inter"], geom["n_routed_experts"],
                     geom["n_group"], geom["topk_group"], geom["top_k"],
                     geom["n_shared_experts"], geom.get("shared_inter", 0),
                     float(geom["routed_scaling_factor"]), WFMT.get(wfmt, wfmt), options,
                     float(geom.get("expert_top_p", 0.0)))


def qexperts(gate, up, down) -> MoeQExperts:
    """Each argument: (q, scale, gscale-or-None) tensors (device tensors; for
    an expert cache's host store, pinned CPU tensors)."""
    def proj(p):
        return MoeQProj(p[0].data_ptr(), p[1].data_ptr(), None if p[2] is None else p[2].data_ptr())
    return MoeQExperts(proj(gate), proj(up), proj(down))


def moe_workspace_size(cfg: MoeConfig, T: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(cfg), T, ctypes.byref(n)), "moe_workspace_size")
    return n.value


def workspace(cfg: MoeConfig, T: int, device="cuda") -> torch.Tensor:
    """A torch-allocated workspace of the size the library asks for."""
    return torch.empty(max(moe_workspace_size(cfg, T), 1), dtype=torch.uint8, device=device)


def moe_route(cfg, T, x, router_w, bias, topk_ids, topk_w, ws, stream=None):
    _check(lib().moe_route(ctypes.byref(cfg), T, _p(x), _p(router_w), _p(bias), _p(topk_ids),
                           _p(topk_w), _p(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "moe_route")


def moe_permute(cfg, T, topk_ids, expert_offsets, sorted_token, inv_perm, active_experts,
                n_active, ws, stream=None):
    _check(lib().moe_permute(ctypes.byref(cfg), T, _p(topk_ids), _p(expert_offsets),
                             _p(sorted_token), _p(inv_perm), _p(active_experts), _p(n_active),
                             _p(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "moe_permute")


def moe_expert_ffn_q4(cfg, T, x, w: MoeQExperts, expert_offsets, sorted_token, active_experts,
                      n_active, out, ws, stream=None):
    _check(lib().moe_expert_ffn_q4(ctypes.byref(cfg), T, _p(x), ctypes.byref(w),
                                   _p(expert_offsets), _p(sorted_token), _p(active_experts),
                                   _p(n_active), _p(out), _p(ws),
                                   0 if ws is None else ws.numel(), _stream(stream)),
           "moe_expert_ffn_q4")


def moe_combine(cfg, T, expert_out, inv_perm, topk_w, shared_out, y, out_dtype=MOE_OUT_F32,
                stream=None):
    _check(lib().moe_combine(ctypes.byref(cfg), T, _p(expert_out), _p(inv_perm), _p(topk_w),
                             _p(shared_out), _p(y), out_dtype, _stream(stream)), "moe_combine")


def moe_layer(cfg, T, x, router_w, bias, routed: MoeQExperts, shared: Optional[MoeQExperts], y,
              out_dtype=MOE_OUT_F32, topk_ids_out=None, topk_w_out=None, ws=None, stream=None):
    _check(lib().moe_layer(ctypes.byref(cfg), T, _p(x), _p(router_w), _p(bias),
                           ctypes.byref(routed), None if shared is None else ctypes.byref(shared),
                           _p(y), out_dtype, _p(topk_ids_out), _p(topk_w_out), _p(ws),
                           0 if ws is None else ws.numel(), _stream(stream)), "moe_layer")


def moe_layer_trace(cfg, T, x, router_w, bias, routed: MoeQExperts, shared: Optional[MoeQExperts],
                    y, trace: MoeTrace, out_dtype=MOE_OUT_F32, topk_ids_out=None, topk_w_out=None,
                    ws=None, stream=None):
    """moe_layer recording kernel-boundary events into `trace` (whose events
    the caller created, e.g. from torch.cuda.Event(enable_timing=True).cuda_event)."""
    _check(lib().moe_layer_trace(ctypes.byref(cfg), T, _p(x), _p(router_w), _p(bias),
                                 ctypes.byref(routed),
                                 None if shared is None else ctypes.byref(shared), _p(y),
                                 out_dtype, _p(topk_ids_out), _p(topk_w_out), _p(ws),
                                 0 if ws is None else ws.numel(), _stream(stream),
                                 ctypes.byref(trace)), "moe_layer_trace")


def moe_layer_flags(ws, stream=None) -> int:
    """MOE_FLAG_* bits raised by the last moe_layer call on workspace `ws`
    (waits for the work queued on `stream`)."""
    f = ctypes.c_uint32(0)
    _check(lib().moe_layer_flags(_p(ws), ctypes.byref(f), _stream(stream)), "moe_layer_flags")
    return f.value


def moe_layer_noalloc(cfg, T, x, router_w, bias, routed: MoeQExperts,
                      shared: Optional[MoeQExperts], y, out_dtype=MOE_OUT_F32, topk_ids_out=None,
                      topk_w_out=None, stream=None):
    """moe_layer on the library's own device workspace (no workspace argument)."""
    _check(lib().moe_layer_noalloc(ctypes.byref(cfg), T, _p(x), _p(router_w), _p(bias),
                                   ctypes.byref(routed),
                                   None if shared is None else ctypes.byref(shared), _p(y),
                                   out_dtype, _p(topk_ids_out), _p(topk_w_out), _stream(stream)),
           "moe_layer_noalloc")


def _id_array(experts):
    arr = (ctypes.c_int32 * max(len(experts), 1))(*[int(e) for e in experts])
    return arr, len(experts)


def moe_cache_create(cfg: MoeConfig, n_slots: int, host_store: MoeQExperts,
                     slots: MoeQExperts) -> ctypes.c_void_p:
    h = ctypes.c_void_p(None)
    _check(lib().moe_cache_create(ctypes.byref(cfg), n_slots, ctypes.byref(host_store),
                                  ctypes.byref(slots), ctypes.byref(h)), "moe_cache_create")
    return h


def moe_cache_destroy(cache) -> None:
    _check(lib().moe_cache_destroy(cache), "moe_cache_destroy")


def moe_layer_cached(cache, T, x, router_w, bias, shared: Optional[MoeQExperts], y,
                     out_dtype=MOE_OUT_F32, topk_ids_out=None, topk_w_out=None, ws=None,
                     stream=None):
    _check(lib().moe_layer_cached(cache, T, _p(x), _p(router_w), _p(bias),
                                  None if shared is None else ctypes.byref(shared), _p(y),
                                  out_dtype, _p(topk_ids_out), _p(topk_w_out), _p(ws),
                                  0 if ws is None else ws.numel(), _stream(stream)),
           "moe_layer_cached")


def moe_cache_prefetch(cache, experts, stream=None) -> int:
    arr, n = _id_array(experts)
    loaded = ctypes.c_int32(0)
    _check(lib().moe_cache_prefetch(cache, arr, n, ctypes.byref(loaded), _stream(stream)),
           "moe_cache_prefetch")
    return loaded.value


def moe_cache_pin(cache, experts, stream=None) -> None:
    arr, n = _id_array(experts)
    _check(lib().moe_cache_pin(cache, arr, n, _stream(stream)), "moe_cache_pin")


def moe_cache_unpin_all(cache) -> None:
    _check(lib().moe_cache_unpin_all(cache), "moe_cache_unpin_all")


def moe_cache_get_stats(cache) -> dict:
    st = MoeCacheStats()
    _check(lib().moe_cache_get_stats(cache, ctypes.byref(st)), "moe_cache_get_stats")
    return {name: getattr(st, name) for name, _ in MoeCacheStats._fields_}


def moe_cache_slot_of(cache, expert: int) -> int:
    s = ctypes.c_int32(0)
    _check(lib().moe_cache_slot_of(cache, expert, ctypes.byref(s)), "moe_cache_slot_of")
    return s.value


# ---- MXFP4 and router-balance operators --------------------------------------
# Sizes, types and strides come from the tensors; one whose shape, type or
# layout does not fit the others, or that does not lie on the current device
# (whose kernels would read another device's memory), raises QmoeError
# (MOE_ERR_INVALID_ARG).
_current_device = torch._C._cuda_getDevice
_several = True     # more than one device; known once the library is loaded
_DT = {torch.float32: MOE_DT_F32, torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16}
_SCORE = {"sigmoid": MOE_SCORE_SIGMOID, "softmax": MOE_SCORE_SOFTMAX}


def _require(ok: bool, where: str):
    if not ok:
        raise QmoeError(MOE_ERR_INVALID_ARG, where)


def _fits(where: str, dev: int, t: torch.Tensor, dtype, shape: tuple):
    """`t` is a contiguous tensor of this type and shape on this device."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()):
        raise QmoeError(MOE_ERR_INVALID_ARG, where)


def _matrix(where: str, dev: int, t: torch.Tensor, dtypes):
    """`t` is a matrix on this device whose rows are contiguous; returns its
    rows, columns and row stride."""
    shape = t.shape
    if not (t.get_device() == dev and len(shape) == 2 and t.dtype in dtypes):
        raise QmoeError(MOE_ERR_INVALID_ARG, where)
    rows, cols = shape
    if t.is_contiguous():
        return rows, cols, max(cols, 1)
    ld, step = t.stride()
    _require((cols <= 1 or step == 1) and (rows <= 1 or ld >= cols), where)
    return rows, cols, ld if rows > 1 else max(cols, 1)


def _queue(where: str, stream, dev: int):
    """The stream's handle, by default the device's current stream.  `dev` has
    to be the current device."""
    if dev < 0 or ((dev > 0 or _several) and dev != _current_device()):
        raise QmoeError(MOE_ERR_INVALID_ARG, where)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def mxfp4_empty(rows: int, cols: int, device="cuda"):
    """Uninitialised MXFP4 storage of a [rows][cols] matrix: (codes, scales)."""
    nb = (cols + 31) // 32
    return (torch.empty(rows, 16 * nb, dtype=torch.uint8, device=device),
            torch.empty(rows, nb, dtype=torch.uint8, device=device))


def _mxfp4_rows(where, x, codes, scales):
    dev = x.get_device()
    rows, cols, ld = _matrix(where, dev, x, _DT)
    nb = (cols + 31) // 32
    _fits(where, dev, codes, torch.uint8, (rows, 16 * nb))
    _fits(where, dev, scales, torch.uint8, (rows, nb))
    return rows, cols, ld, dev


def moe_mxfp4_quantize(src, codes, scales, stream=None):
    """Rows of `src` (fp32, bf16 or fp16) to MXFP4 codes and scales."""
    where = "moe_mxfp4_quantize"
    rows, cols, ld, dev = _mxfp4_rows(where, src, codes, scales)
    queue = _queue(where, stream, dev)
    _check(lib().moe_mxfp4_quantize(src.data_ptr(), _DT[src.dtype], rows, cols, ld, codes.data_ptr(),
                                    scales.data_ptr(), queue), where)


def moe_mxfp4_dequantize(codes, scales, dst, stream=None):
    """The values of MXFP4 rows, into `dst` (fp32, bf16 or fp16)."""
    where = "moe_mxfp4_dequantize"
    rows, cols, ld, dev = _mxfp4_rows(where, dst, codes, scales)
    queue = _queue(where, stream, dev)
    _check(lib().moe_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, dst.data_ptr(),
                                      _DT[dst.dtype], ld, queue), where)


def _grouped_weights(where, dev, w_codes, w_scales, expert_offsets):
    shape = w_codes.shape
    _require(len(shape) == 3, where)
    E, N, kb = shape
    _fits(where, dev, w_codes, torch.uint8, shape)
    _fits(where, dev, w_scales, torch.uint8, (E, N, kb // 16))
    if expert_offsets is not None:
        _fits(where, dev, expert_offsets, torch.int32, (E + 1,))
    return E, N, kb * 2


_OUT_DT = (torch.float32, torch.bfloat16)
_BF16 = (torch.bfloat16,)


def moe_mxfp4_matmul(a, w_codes, w_scales, out, a_scale=None, expert_offsets=None, row_index=None,
                     stream=None):
    """out[r] = a[row_index[r]] @ W[expert of r].T over MXFP4 weights [E][n][k/2];
    `a` is bf16 [rows][k], or MXFP4 codes uint8 [rows][k/2] with `a_scale`."""
    where = "moe_mxfp4_matmul"
    dev = out.get_device()
    E, N, K = _grouped_weights(where, dev, w_codes, w_scales, expert_offsets)
    R, cols, ldo = _matrix(where, dev, out, _OUT_DT)
    _require(cols == N, where)
    if a_scale is None:
        a_rows, cols, lda = _matrix(where, dev, a, _BF16)
        _require(cols == K, where)
        dt = MOE_DT_BF16
    else:
        a_rows = a.shape[0]
        _fits(where, dev, a, torch.uint8, (a_rows, K // 2))
        _fits(where, dev, a_scale, torch.uint8, (a_rows, K // 32))
        lda, dt = K, MOE_DT_MXFP4
    if row_index is not None:
        _fits(where, dev, row_index, torch.int32, (R,))
    queue = _queue(where, stream, dev)
    cfg = MoeMatmulConfig(R, N, K, E, a_rows, dt, _DT[out.dtype], lda, ldo)
    _check(lib().moe_mxfp4_matmul(ctypes.byref(cfg), a.data_ptr(), _at(a_scale), w_codes.data_ptr(),
                                  w_scales.data_ptr(), _at(expert_offsets), _at(row_index),
                                  out.data_ptr(), queue), where)


def moe_mxfp4_matmul_dx(dy, w_codes, w_scales, dx, expert_offsets=None, stream=None):
    """dx[r] = dy[r] @ W[expert of r]: the gradient of moe_mxfp4_matmul's rows."""
    where = "moe_mxfp4_matmul_dx"
    dev = dx.get_device()
    E, N, K = _grouped_weights(where, dev, w_codes, w_scales, expert_offsets)
    rows, cols, lda = _matrix(where, dev, dy, _BF16)
    R, dx_cols, ldo = _matrix(where, dev, dx, _OUT_DT)
    _require(rows == R and cols == N and dx_cols == K, where)
    queue = _queue(where, stream, dev)
    cfg = MoeMatmulConfig(R, N, K, E, R, MOE_DT_BF16, _DT[dx.dtype], lda, ldo)
    _check(lib().moe_mxfp4_matmul_dx(ctypes.byref(cfg), dy.data_ptr(), w_codes.data_ptr(),
                                     w_scales.data_ptr(), _at(expert_offsets), dx.data_ptr(), queue),
           where)


def make_balance_config(tokens: int, n_experts: int, top_k: int = 1, n_seq: int = 1,
                        score: str = "sigmoid", dtype=torch.float32,
                        coef: float = 1.0) -> MoeBalanceConfig:
    return MoeBalanceConfig(tokens, n_experts, top_k, n_seq, _SCORE.get(score, score), _DT[dtype], coef)


def moe_balance_workspace_size(cfg: MoeBalanceConfig) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_balance_workspace_size(ctypes.byref(cfg), ctypes.byref(n)),
           "moe_balance_workspace_size")
    return n.value


def balance_workspace(tokens: int, n_experts: int, n_seq: int = 1, device="cuda") -> torch.Tensor:
    """A torch-allocated workspace for moe_balance_loss of this size."""
    n = moe_balance_workspace_size(make_balance_config(tokens, n_experts, n_seq=n_seq))
    return torch.empty(n, dtype=torch.uint8, device=device)


def _balance(where, stream, logits, topk_ids, counts, tokens, coef, score, seq_offsets):
    _require(logits.dim() == 2 and topk_ids.dim() == 2 and counts.dim() == 2 and score in _SCORE, where)
    dev = counts.get_device()
    queue = _queue(where, stream, dev)
    T, E = shape = logits.shape
    S, K = counts.shape[0], topk_ids.shape[1]
    _require(logits.dtype in _OUT_DT, where)
    _fits(where, dev, logits, logits.dtype, shape)
    _fits(where, dev, topk_ids, torch.int32, (T, K))
    _fits(where, dev, counts, torch.int32, (S, E))
    _fits(where, dev, tokens, torch.int32, (S,))
    if seq_offsets is not None:
        _fits(where, dev, seq_offsets, torch.int32, (S + 1,))
    return MoeBalanceConfig(T, E, K, S, _SCORE[score], _DT[logits.dtype], coef), dev, queue


def moe_balance_loss(logits, topk_ids, counts, tokens, loss, coef, score="sigmoid", seq_offsets=None,
                     ws=None, stream=None):
    """The router's balance loss (loss [1]), its picks per sequence and expert
    (counts [S][E]) and routed tokens per sequence (tokens [S]).  Without `ws`
    the call takes a workspace from torch's allocator, on its stream."""
    where = "moe_balance_loss"
    cfg, dev, queue = _balance(where, stream, logits, topk_ids, counts, tokens, coef, score, seq_offsets)
    _fits(where, dev, loss, torch.float32, (1,))
    if ws is None:
        # of the memory that belongs to the call's stream, whose order keeps it until the call has run
        with torch.cuda.stream(torch.cuda.ExternalStream(queue) if queue else torch.cuda.default_stream()):
            ws = torch.empty(moe_balance_workspace_size(cfg), dtype=torch.uint8, device=counts.device)
    else:
        _require(ws.get_device() == dev and ws.dtype is torch.uint8 and ws.is_contiguous(), where)
    _check(lib().moe_balance_loss(ctypes.byref(cfg), logits.data_ptr(), topk_ids.data_ptr(),
                                  _at(seq_offsets), counts.data_ptr(), tokens.data_ptr(),
                                  loss.data_ptr(), ws.data_ptr(), ws.numel(), queue), where)


def moe_balance_loss_grad(logits, topk_ids, counts, tokens, dlogits, coef, score="sigmoid",
                          seq_offsets=None, dloss=None, stream=None):
    """dlogits [T][E]: dloss (1 if None) times the loss's gradient, from the
    counts and tokens that moe_balance_loss wrote."""
    where = "moe_balance_loss_grad"
    cfg, dev, queue = _balance(where, stream, logits, topk_ids, counts, tokens, coef, score, seq_offsets)
    _fits(where, dev, dlogits, logits.dtype, logits.shape)
    if dloss is not None:
        _fits(where, dev, dloss, torch.float32, (1,))
    _check(lib().moe_balance_loss_grad(ctypes.byref(cfg), logits.data_ptr(), topk_ids.data_ptr(),
                                       _at(seq_offsets), counts.data_ptr(), tokens.data_ptr(),
                                       _at(dloss), dlogits.data_ptr(), queue), where)


# ---- row operators -------------------------------------------------------------
# Matrices in 8 bits are torch.float8_e4m3fn with fp32 scales [rows], in MXFP4
# uint8 codes with uint8 scales (mxfp4_empty).  Arguments as above.  A call of a
# few rows costs what its checks cost, so each reads a tensor's properties once
# and the C structs are packed.
_E4M3, _U8, _I32, _F32 = torch.float8_e4m3fn, torch.uint8, torch.int32, torch.float32
_PLAIN = {torch.float32: MOE_DT_F32, torch.bfloat16: MOE_DT_BF16}


def _packer(config):
    """bytes of a ctypes struct of int32, float and int64 fields from their values."""
    code = {ctypes.c_int32: "i", ctypes.c_float: "f", ctypes.c_int64: "q"}
    s = struct.Struct("@" + "".join(code[t] for _, t in config._fields_))
    assert s.size == ctypes.sizeof(config)
    floats = [i for i, (_, t) in enumerate(config._fields_) if t is ctypes.c_float]

    def pack(*values):
        try:
            return s.pack(*values)
        except (struct.error, OverflowError):
            pass
        try:                                       # no number, or one past fp32
            struct.pack("f" * len(floats), *(values[i] for i in floats))
        except (struct.error, OverflowError):
            raise QmoeError(MOE_ERR_INVALID_ARG, config.__name__) from None
        raise QmoeError(MOE_ERR_UNSUPPORTED, config.__name__)      # sizes past 32 bits
    return pack


_norm_config, _norm_grad_config = _packer(MoeRmsnormConfig), _packer(MoeRmsnormGradConfig)
_rows_config, _swiglu_config = _packer(MoeRowsConfig), _packer(MoeSwigluConfig)


def _plain(where: str, dev: int, t: torch.Tensor):
    """dtype, rows, columns and row stride of an fp32 or bf16 matrix on this device
    whose rows are contiguous."""
    dt, shape = _PLAIN.get(t.dtype), t.shape
    if dt is None or len(shape) != 2 or t.get_device() != dev:
        raise QmoeError(MOE_ERR_INVALID_ARG, where)
    rows, cols = shape
    if t.is_contiguous():
        return dt, rows, cols, cols or 1
    ld, step = t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and ld < cols):
        raise QmoeError(MOE_ERR_INVALID_ARG, where)
    return dt, rows, cols, ld if rows > 1 else cols or 1


def _weight(where, dev, w, cols):
    dt = _PLAIN.get(w.dtype)
    if dt is None or w.shape != (cols,) or w.get_device() != dev or not w.is_contiguous():
        raise QmoeError(MOE_ERR_INVALID_ARG, where)
    return dt


def _coded(where, dev, codes, scale, rows, cols):
    """dtype of a matrix in 8 or 4 bits of this size, with its scales."""
    _require(scale is not None, where)
    if codes.dtype is _E4M3:
        _fits(where, dev, codes, _E4M3, (rows, cols))
        _fits(where, dev, scale, _F32, (rows,))
        return MOE_DT_E4M3
    nb = (cols + 31) // 32
    _fits(where, dev, codes, _U8, (rows, 16 * nb))
    _fits(where, dev, scale, _U8, (rows, nb))
    return MOE_DT_MXFP4


def moe_rmsnorm(x, weight, eps, y=None, residual=None, h=None, q=None, q_scale=None, stream=None):
    """h = x + residual (h = x without one) and y = h / sqrt(mean(h^2) + eps) * weight
    over the rows of `x`; `q` with `q_scale` takes y in E4M3 or MXFP4.  h may be
    `residual` itself."""
    where = "moe_rmsnorm"
    dev = x.get_device()
    queue = _queue(where, stream, dev)
    xt, rows, cols, ldx = _plain(where, dev, x)
    wt = _weight(where, dev, weight, cols)
    size = rows, cols
    rt = yt = qt = ldr = ldh = ldy = 0
    rp = hp = yp = qp = sp = None
    if residual is not None:
        rt, r, c, ldr = _plain(where, dev, residual)
        _require((r, c) == size, where)
        rp = residual.data_ptr()
    if h is not None:
        ht, r, c, ldh = _plain(where, dev, h)
        _require((r, c) == size and rp is not None and ht == rt, where)
        hp = h.data_ptr()
    if y is not None:
        yt, r, c, ldy = _plain(where, dev, y)
        _require((r, c) == size, where)
        yp = y.data_ptr()
    if q is not None:
        qt = _coded(where, dev, q, q_scale, rows, cols)
        qp = q.data_ptr()
    if q_scale is not None:
        sp = q_scale.data_ptr()
    status = lib().moe_rmsnorm(_norm_config(rows, cols, xt, rt, wt, yt, qt, eps, ldx, ldr, ldh, ldy), x.data_ptr(), rp,
                               weight.data_ptr(), hp, yp, qp, sp, queue)
    if status:
        raise QmoeError(status, where)


def moe_rmsnorm_workspace_size(rows: int, cols: int) -> int:
    where = "moe_rmsnorm_workspace_size"
    if max(rows, cols) >= 1 << 31:           # ctypes would cut them to 32 bits
        raise QmoeError(MOE_ERR_UNSUPPORTED, where)
    _require(min(rows, cols) >= 0, where)
    n = ctypes.c_size_t(0)
    _check(lib().moe_rmsnorm_workspace_size(rows, cols, ctypes.byref(n)), where)
    return n.value


def rmsnorm_workspace(rows: int, cols: int, device="cuda") -> torch.Tensor:
    """A torch-allocated workspace for moe_rmsnorm_grad of this size."""
    return torch.empty(moe_rmsnorm_workspace_size(rows, cols), dtype=torch.uint8, device=device)


def moe_rmsnorm_grad(dy, h, weight, eps, dx, dh=None, dweight=None, ws=None, stream=None):
    """dx: the gradient of moe_rmsnorm's x and residual, from the h that it wrote
    (x without a residual), plus `dh`; dweight fp32 [cols].  Without `ws` a call
    with dweight takes a workspace from torch's allocator, on its stream."""
    where = "moe_rmsnorm_grad"
    dev = dx.get_device()
    queue = _queue(where, stream, dev)
    xt, rows, cols, lddx = _plain(where, dev, dx)
    ht, r, c, ldh = _plain(where, dev, h)
    yt, r2, c2, lddy = _plain(where, dev, dy)
    _require(r == r2 == rows and c == c2 == cols, where)
    wt = _weight(where, dev, weight, cols)
    lddh = n = 0
    dp = wp = sp = None
    if dh is not None:
        dt, r, c, lddh = _plain(where, dev, dh)
        _require(dt == xt and r == rows and c == cols, where)
        dp = dh.data_ptr()
    if dweight is not None:
        _fits(where, dev, dweight, _F32, (cols,))
        wp = dweight.data_ptr()
        if ws is None:
            # of the memory that belongs to the call's stream, whose order keeps it until the call has run
            with torch.cuda.stream(torch.cuda.ExternalStream(queue) if queue else torch.cuda.default_stream()):
                ws = torch.empty(moe_rmsnorm_workspace_size(rows, cols), dtype=torch.uint8, device=dx.device)
    if ws is not None:
        _require(ws.get_device() == dev and ws.dtype is _U8 and ws.is_contiguous(), where)
        n, sp = ws.numel(), ws.data_ptr()
    status = lib().moe_rmsnorm_grad(_norm_grad_config(rows, cols, ht, wt, yt, xt, eps, ldh, lddy, lddh, lddx), dy.data_ptr(),
                                    h.data_ptr(), weight.data_ptr(), dp, dx.data_ptr(), wp, sp, n, queue)
    if status:
        raise QmoeError(status, where)


def _picks(where, dev, inv_perm, tokens, weights=None):
    """Picks a token; `weights` (if any) fit them."""
    shape = inv_perm.shape
    if len(shape) != 2 or shape[0] != tokens:
        raise QmoeError(MOE_ERR_INVALID_ARG, where)
    _fits(where, dev, inv_perm, _I32, shape)
    if weights is not None:
        _fits(where, dev, weights, _F32, shape)
    return shape[1]


def moe_dispatch(x, inv_perm, rows, x_scale=None, row_scale=None, stream=None):
    """rows[inv_perm[t, i]] = x[t]; picks outside [0, rows) take no row.  `x` and
    `rows` are fp32 or bf16, or both in E4M3 or MXFP4 with their scales."""
    where = "moe_dispatch"
    dev = rows.get_device()
    queue = _queue(where, stream, dev)
    xs = rs = None
    if x.dtype in _PLAIN:
        tt, T, cols, ldt = _plain(where, dev, x)
        rt, slots, rcols, ldr = _plain(where, dev, rows)
        _require(cols == rcols and x_scale is None and row_scale is None, where)
    else:
        _require(x.dim() == 2 and rows.dim() == 2 and rows.dtype is x.dtype, where)
        T, slots = x.shape[0], rows.shape[0]
        # of MXFP4 rows the last block counts whole: columns only say how many blocks there are
        cols = ldt = ldr = x.shape[1] * (1 if x.dtype is _E4M3 else 2)
        tt = _coded(where, dev, x, x_scale, T, cols)
        rt = _coded(where, dev, rows, row_scale, slots, cols)
        xs, rs = x_scale.data_ptr(), row_scale.data_ptr()
    K = _picks(where, dev, inv_perm, T)
    status = lib().moe_dispatch(_rows_config(T, cols, K, slots, tt, rt, 0, ldt, ldr, 0), x.data_ptr(), xs, inv_perm.data_ptr(),
                                rows.data_ptr(), rs, queue)
    if status:
        raise QmoeError(status, where)


def moe_collect(rows, inv_perm, y, weights=None, addend=None, stream=None):
    """y[t] = addend[t] + sum_i weights[t, i] * rows[inv_perm[t, i]]; picks outside
    [0, rows) count for nothing.  The gradient of moe_dispatch is this call without
    weights.  `addend` may be y itself."""
    where = "moe_collect"
    dev = y.get_device()
    queue = _queue(where, stream, dev)
    yt, T, cols, ldt = _plain(where, dev, y)
    rt, slots, rcols, ldr = _plain(where, dev, rows)
    K = _picks(where, dev, inv_perm, T, weights)
    at = lda = 0
    ap = None
    if addend is not None:
        at, r, c, lda = _plain(where, dev, addend)
        _require(r == T and c == cols, where)
        ap = addend.data_ptr()
    _require(cols == rcols, where)
    status = lib().moe_collect(_rows_config(T, cols, K, slots, yt, rt, at, ldt, ldr, lda), rows.data_ptr(), inv_perm.data_ptr(),
                               None if weights is None else weights.data_ptr(), ap, y.data_ptr(), queue)
    if status:
        raise QmoeError(status, where)


def moe_collect_grad(dy, inv_perm, drows=None, weights=None, rows=None, dweights=None, stream=None):
    """Gradient of moe_collect by its rows (drows[inv_perm[t, i]] = weights[t, i] *
    dy[t]; rows of no pick are left as they are) and by its weights (dweights[t, i] =
    dy[t] . rows[inv_perm[t, i]], 0 for picks without a row).  drows may be `rows`
    itself."""
    where = "moe_collect_grad"
    dev = dy.get_device()
    queue = _queue(where, stream, dev)
    yt, T, cols, ldt = _plain(where, dev, dy)
    K = _picks(where, dev, inv_perm, T, weights)
    like = drows if rows is None else rows
    _require(like is not None, where)
    rt, slots, rcols, ldr = _plain(where, dev, like)
    _require(cols == rcols, where)
    rp = wp = None
    if rows is not None:
        rp = rows.data_ptr()
        if drows is not None:
            dt, r, c, ld = _plain(where, dev, drows)
            _require(dt == rt and r == slots and c == cols and ld == ldr, where)
    if dweights is not None:
        _require(rp is not None, where)
        _fits(where, dev, dweights, _F32, (T, K))
        wp = dweights.data_ptr()
    status = lib().moe_collect_grad(_rows_config(T, cols, K, slots, yt, rt, 0, ldt, ldr, 0), dy.data_ptr(), rp,
                                    inv_perm.data_ptr(), None if weights is None else weights.data_ptr(),
                                    None if drows is None else drows.data_ptr(), wp, queue)
    if status:
        raise QmoeError(status, where)


def _experts(where, dev, expert_offsets):
    """Experts of a table of offsets; without one every row counts."""
    if expert_offsets is None:
        return 1
    shape = expert_offsets.shape
    _require(len(shape) == 1 and shape[0] >= 2, where)
    _fits(where, dev, expert_offsets, _I32, shape)
    return shape[0] - 1


def moe_swiglu(gu, out, out_scale=None, expert_offsets=None, stream=None):
    """out = silu(gate) * up over rows [gate | up]; `out` fp32, bf16, or E4M3 or
    MXFP4 with `out_scale`.  Rows from expert_offsets[-1] on are left as they are."""
    where = "moe_swiglu"
    dev = gu.get_device()
    queue = _queue(where, stream, dev)
    gt, rows, twice, ldg = _plain(where, dev, gu)
    cols = twice >> 1
    sp = None
    if out.dtype in _PLAIN:
        ot, r, c, ldo = _plain(where, dev, out)
        _require(r == rows and 2 * c == twice and out_scale is None, where)
    else:
        _require(2 * cols == twice, where)
        ot, ldo = _coded(where, dev, out, out_scale, rows, cols), cols
        sp = out_scale.data_ptr()
    E = _experts(where, dev, expert_offsets)
    status = lib().moe_swiglu(_swiglu_config(rows, cols, E, gt, ot, ldg, ldo), gu.data_ptr(),
                              None if expert_offsets is None else expert_offsets.data_ptr(), out.data_ptr(), sp, queue)
    if status:
        raise QmoeError(status, where)


def moe_swiglu_grad(gu, dh, dgu, expert_offsets=None, stream=None):
    """dgu: the gradient of moe_swiglu's gate and up from that of its output.  dgu may
    be `gu` itself."""
    where = "moe_swiglu_grad"
    dev = gu.get_device()
    queue = _queue(where, stream, dev)
    gt, rows, twice, ldg = _plain(where, dev, gu)
    ht, r, cols, ldo = _plain(where, dev, dh)
    dt, r2, c2, ld = _plain(where, dev, dgu)
    _require(r == r2 == rows and twice == c2 == 2 * cols and dt == gt and ld == ldg, where)
    E = _experts(where, dev, expert_offsets)
    status = lib().moe_swiglu_grad(_swiglu_config(rows, cols, E, gt, ht, ldg, ldo), gu.data_ptr(), dh.data_ptr(),
                                   None if expert_offsets is None else expert_offsets.data_ptr(), dgu.data_ptr(), queue)
    if status:
        raise QmoeError(status, where)

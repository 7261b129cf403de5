"""ctypes binding of libmoert.so: the C-ABI calls under the same names.

Argument marshalling only: tensors become device pointers, torch streams
become hipStream_t handles, statuses become exceptions (the operators without
a context also take sizes and strides from their tensors, and check them).  Every step of the
MoE layer runs in the library's HIP kernels and host code.  torch is imported
first so the library binds to the HIP runtime torch already loaded (both
carry the SONAME libamdhip64.so.7): one runtime per process.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch  # noqa: F401  (loads the process's HIP runtime before libmoert)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoert.so")

MOE_OK, MOE_EINVAL, MOE_ENOMEM, MOE_ENOSPC, MOE_EHIP, MOE_EBUSY, MOE_ETIMEDOUT, \
    MOE_EUNSUPPORTED = 0, -1, -2, -3, -4, -5, -6, -7
MOE_F32, MOE_BF16, MOE_MXFP4, MOE_F8 = 0, 1, 2, 3
MOE_HYBRID, MOE_OFFLOAD, MOE_CPU = 0, 1, 2
DTYPES = {"f32": MOE_F32, "bf16": MOE_BF16, "mxfp4": MOE_MXFP4}


class MoeConfig(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("w_dtype", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("n_slots", ctypes.c_int32), ("max_slots", ctypes.c_int32),
                ("max_tokens", ctypes.c_int32), ("bw_pcie_mbps", ctypes.c_int64),
                ("bw_host_mbps", ctypes.c_int64), ("max_fetch", ctypes.c_int32),
                ("mode", ctypes.c_int32), ("cpu_threads", ctypes.c_int32),
                ("max_prefill_tokens", ctypes.c_int32), ("timing", ctypes.c_int32)]


class PlanCounts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("n_uniq", "n_hit", "n_miss", "q", "n_cpu", "n_gpu", "K", "tick_lo")]


class PlanView(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("uniq", ctypes.c_void_p), ("hits", ctypes.c_void_p),
                ("misses", ctypes.c_void_p), ("victims", ctypes.c_void_p),
                ("fill_u", ctypes.c_void_p), ("fill_slot", ctypes.c_void_p),
                ("fill_old", ctypes.c_void_p), ("cpu_u", ctypes.c_void_p),
                ("gpu_u", ctypes.c_void_p), ("gpu_slot", ctypes.c_void_p),
                ("slot_map", ctypes.c_void_p), ("id2slot", ctypes.c_void_p),
                ("slot2id", ctypes.c_void_p), ("slot_ts", ctypes.c_void_p),
                ("tick", ctypes.c_void_p), ("p_gpu", ctypes.c_void_p), ("p_cpu", ctypes.c_void_p),
                ("slot_base", ctypes.c_void_p), ("n_slots", ctypes.c_int32),
                ("max_slots", ctypes.c_int32), ("umax", ctypes.c_int32), ("kmax", ctypes.c_int32),
                ("h_marked", ctypes.c_void_p)]


class PrefillView(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p),
                ("tiles", ctypes.c_void_p), ("hmid", ctypes.c_void_p), ("prow", ctypes.c_void_p),
                ("n_experts", ctypes.c_int32), ("max_pairs", ctypes.c_int32),
                ("max_tiles", ctypes.c_int32)]


class Stats(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int32), ("occupied", ctypes.c_int32),
                ("plans", ctypes.c_int64), ("hits", ctypes.c_int64), ("fills", ctypes.c_int64),
                ("cpu", ctypes.c_int64), ("evictions", ctypes.c_int64),
                ("prefill_layers", ctypes.c_int64), ("resizes", ctypes.c_int64),
                ("prefill_h2d_experts", ctypes.c_int64), ("prefill_d2d_experts", ctypes.c_int64)]


PHASES = ("route", "plan", "fill", "ffn", "merge", "host", "prefill_copy", "prefill_group",
          "prefill_gemm", "prefill_merge")


class Timing(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_int64 * len(PHASES)), ("ms", ctypes.c_double * len(PHASES))]

    def as_dict(self):
        return {p: dict(calls=self.calls[i], ms=self.ms[i]) for i, p in enumerate(PHASES)}


class GroupedArgs(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("n_rows", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32),
                ("y_dtype", ctypes.c_int32), ("glu", ctypes.c_int32), ("x", ctypes.c_void_p),
                ("x_scales", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("n_x", ctypes.c_int32),
                ("x_index_div", ctypes.c_int32), ("x_index", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("w_scales", ctypes.c_void_p), ("w_stride", ctypes.c_int64),
                ("ws_stride", ctypes.c_int64), ("offsets", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("ldy", ctypes.c_int64), ("n_y", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("y_index", ctypes.c_void_p)]


class CombineNormArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("p", "w", "ids", "residual", "out", "post_weight", "gate", "weight", "y", "y_scales")] + \
               [(n, ctypes.c_int64) for n in ("ldp", "ldres", "ldout", "ldg", "ldy", "T")] + \
               [(n, ctypes.c_int32) for n in
                ("k", "H", "n_experts", "gate_cols", "p_dtype", "residual_dtype", "out_dtype", "post_dtype",
                 "gate_dtype", "weight_dtype", "y_dtype", "reserved")] + \
               [("scale", ctypes.c_float), ("eps", ctypes.c_float)]


class MoertError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({_strerror(status)}): {detail}")


_lib = None


def lib():
    """Load libmoert.so; fails loudly when the HIP library has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build the HIP library first "
                "(python -m routed_expert_execution_moe_amd.build or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        f32 = ctypes.c_float
        cfgp = ctypes.POINTER(MoeConfig)
        sig = {
            "moe_expert_bytes": ([cfgp], sz),
            "moe_host_pool_alloc": ([sz, ctypes.POINTER(vp)], i32),
            "moe_host_pool_free": ([vp], i32),
            "moe_create": ([cfgp, vp, sz, ctypes.POINTER(vp)], i32),
            "moe_destroy": ([vp], i32),
            "moe_route_topk": ([vp, vp, i32, vp, vp, vp], i32),
            "moe_cache_plan": ([vp, i32, vp, i32, vp, vp], i32),
            "moe_expert_ffn": ([vp, i32, vp, i32, vp], i32),
            "moe_merge": ([vp, vp, i32, vp, vp], i32),
            "moe_cache_resize": ([vp, i32, i32], i32),
            "moe_measure_bandwidth": ([vp, i32, i32, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                      ctypes.POINTER(i64)], i32),
            "moe_recommend_mode": ([i64, i64, ctypes.c_double, ctypes.POINTER(i32)], i32),
            "moe_set_split": ([vp, i64, i64, i32], i32),
            "moe_prefill_set_buffers": ([vp, i32], i32),
            "moe_set_cpu_layers": ([vp, ctypes.POINTER(ctypes.c_uint8), i32], i32),
            "moe_prefill_layer": ([vp, i32, vp, i32, vp, vp, vp, vp], i32),
            "moe_prefill_layer_noalloc": ([vp, i32, vp, i32, vp, vp, vp, vp], i32),
            "moe_plan_view_get": ([vp, ctypes.POINTER(PlanView)], i32),
            "moe_prefill_view_get": ([vp, ctypes.POINTER(PrefillView)], i32),
            "moe_ctx_stats": ([vp, ctypes.POINTER(Stats)], i32),
            "moe_ctx_timing": ([vp, ctypes.POINTER(Timing), i32], i32),
            "moe_mx_quantize": ([vp, i32, i64, i32, i64, vp, vp, vp], i32),
            "moe_mx_dequantize": ([vp, vp, i64, i32, vp, i32, i64, vp], i32),
            "moe_mx_gemm": ([vp, i32, vp, i64, vp, vp, vp, i32, i64, i32, i32, i32, vp], i32),
            "moe_f8_quantize": ([vp, i32, i32, i64, i32, i64, i64, i32, vp, vp, vp], i32),
            "moe_f8_dequantize": ([vp, vp, i32, i64, i32, i32, vp, i32, i64, i64, vp], i32),
            "moe_f8_gemm": ([vp, vp, i64, vp, vp, vp, i32, i64, i32, i32, i32, vp], i32),
            "moe_norm": ([vp, i32, i64, vp, i32, f32, i64, i32, vp, i32, vp, i64, vp], i32),
            "moe_combine_norm": ([vp, vp], i32),
            "moe_group_workspace": ([i32, i32, i32], sz),
            "moe_group_pairs": ([vp, i32, i32, i32, vp, vp, vp, sz, vp], i32),
            "moe_grouped_gemm": ([ctypes.POINTER(GroupedArgs), vp], i32),
            "moe_combine_pairs": ([vp, i32, i64, vp, vp, i32, i32, i32, i32, vp, i32, i64, vp], i32),
            "moe_strerror": ([i32], ctypes.c_char_p),
            "moe_last_error": ([], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _strerror(s: int) -> str:
    return lib().moe_strerror(s).decode()


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoertError(status, where, lib().moe_last_error().decode())


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> int | None:
    if s is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def config(L, E, k, H, I, w_dtype, act_dtype, n_slots, max_slots=None, max_tokens=1,
           bw_pcie_mbps=1, bw_host_mbps=1, max_fetch=0, mode=MOE_HYBRID, cpu_threads=0,
           max_prefill_tokens=0, timing=0) -> MoeConfig:
    return MoeConfig(L, E, k, H, I, DTYPES.get(w_dtype, w_dtype), DTYPES.get(act_dtype, act_dtype),
                     n_slots, n_slots if max_slots is None else max_slots, max_tokens,
                     bw_pcie_mbps, bw_host_mbps, max_fetch, mode, cpu_threads, max_prefill_tokens,
                     timing)


# ------------------------------------------------------------------ the C-ABI calls
def moe_expert_bytes(cfg: MoeConfig) -> int:
    return lib().moe_expert_bytes(ctypes.byref(cfg))


def moe_host_pool_alloc(nbytes: int) -> int:
    p = ctypes.c_void_p()
    _check(lib().moe_host_pool_alloc(nbytes, ctypes.byref(p)), "moe_host_pool_alloc")
    return p.value


def moe_host_pool_free(addr: int) -> None:
    _check(lib().moe_host_pool_free(addr), "moe_host_pool_free")


def moe_create(cfg: MoeConfig, host_pool: int, host_pool_bytes: int) -> int:
    out = ctypes.c_void_p()
    _check(lib().moe_create(ctypes.byref(cfg), host_pool, host_pool_bytes, ctypes.byref(out)),
           "moe_create")
    return out.value


def moe_destroy(ctx: int) -> None:
    _check(lib().moe_destroy(ctx), "moe_destroy")


def moe_route_topk(ctx, logits, T, ids, w, stream=None):
    _check(lib().moe_route_topk(ctx, _ptr(logits), T, _ptr(ids), _ptr(w), _stream(stream)),
           "moe_route_topk")


def moe_cache_plan(ctx, layer, ids, T, x, stream=None):
    _check(lib().moe_cache_plan(ctx, layer, _ptr(ids), T, _ptr(x), _stream(stream)),
           "moe_cache_plan")


def moe_expert_ffn(ctx, layer, x, T, stream=None):
    _check(lib().moe_expert_ffn(ctx, layer, _ptr(x), T, _stream(stream)), "moe_expert_ffn")


def moe_merge(ctx, w, T, y, stream=None):
    _check(lib().moe_merge(ctx, _ptr(w), T, _ptr(y), _stream(stream)), "moe_merge")


def moe_cache_resize(ctx, new_n_slots, timeout_ms=300_000):
    _check(lib().moe_cache_resize(ctx, new_n_slots, timeout_ms), "moe_cache_resize")


def moe_measure_bandwidth(ctx, n_experts=8, reps=5, h2d=False):
    """(B_P, B_H) in MB/s, measured on the context's expert shape; with
    h2d=True also the pinned host-to-device copy rate: (B_P, B_H, B_H2D)."""
    bp, bh, bc = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().moe_measure_bandwidth(ctx, n_experts, reps, ctypes.byref(bp), ctypes.byref(bh),
                                       ctypes.byref(bc) if h2d else None), "moe_measure_bandwidth")
    return (bp.value, bh.value, bc.value) if h2d else (bp.value, bh.value)


def moe_recommend_mode(bw_pcie_mbps, bw_host_mbps, threshold=2.0):
    m = ctypes.c_int32()
    _check(lib().moe_recommend_mode(bw_pcie_mbps, bw_host_mbps, threshold, ctypes.byref(m)),
           "moe_recommend_mode")
    return m.value


def moe_set_cpu_layers(ctx, flags):
    """flags: sequence of L truthy values (layers that decode on the host), or None."""
    if flags is None:
        _check(lib().moe_set_cpu_layers(ctx, None, 0), "moe_set_cpu_layers")
        return
    arr = (ctypes.c_uint8 * len(flags))(*[1 if f else 0 for f in flags])
    _check(lib().moe_set_cpu_layers(ctx, arr, len(flags)), "moe_set_cpu_layers")


def moe_set_split(ctx, bw_pcie_mbps, bw_host_mbps, mode):
    _check(lib().moe_set_split(ctx, bw_pcie_mbps, bw_host_mbps, mode), "moe_set_split")


def moe_prefill_set_buffers(ctx, n_buffers):
    _check(lib().moe_prefill_set_buffers(ctx, n_buffers), "moe_prefill_set_buffers")


def moe_prefill_layer(ctx, layer, x, T, ids, w, y, stream=None):
    _check(lib().moe_prefill_layer(ctx, layer, _ptr(x), T, _ptr(ids), _ptr(w), _ptr(y),
                                   _stream(stream)), "moe_prefill_layer")


def moe_prefill_layer_noalloc(ctx, layer, x, T, ids, w, y, stream=None):
    _check(lib().moe_prefill_layer_noalloc(ctx, layer, _ptr(x), T, _ptr(ids), _ptr(w), _ptr(y),
                                           _stream(stream)), "moe_prefill_layer_noalloc")


def moe_plan_view_get(ctx) -> PlanView:
    v = PlanView()
    _check(lib().moe_plan_view_get(ctx, ctypes.byref(v)), "moe_plan_view_get")
    return v


def moe_prefill_view_get(ctx) -> PrefillView:
    v = PrefillView()
    _check(lib().moe_prefill_view_get(ctx, ctypes.byref(v)), "moe_prefill_view_get")
    return v


def moe_ctx_stats(ctx) -> Stats:
    s = Stats()
    _check(lib().moe_ctx_stats(ctx, ctypes.byref(s)), "moe_ctx_stats")
    return s


def moe_ctx_timing(ctx, reset=False) -> dict:
    t = Timing()
    _check(lib().moe_ctx_timing(ctx, ctypes.byref(t), 1 if reset else 0), "moe_ctx_timing")
    return t.as_dict()


# ------------------------------------------------------------------ operators without a context
# Sizes, dtypes and strides come from the tensors, so these also check what the
# library cannot see: shapes that belong together, element types, contiguous
# rows and one device.  The call is made with the tensors' device current, on
# `stream` or on that device's current stream.  The checks are host time in
# front of kernels of a few microseconds: contiguous tensors, the usual case,
# pass _matrix and _whole in a few attribute reads, and only what does not is
# looked at for the reason.  They serve inference: they write their outputs through
# plain pointers and record nothing for autograd, whatever requires a gradient.
# Tensors used on a `stream` other than the one they were allocated on are the
# caller's to order and to keep (torch.Tensor.record_stream), as with any kernel.
_FLOATS = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_U8, _I32, _BF16, _F32 = (torch.uint8,), (torch.int32,), (torch.bfloat16,), (torch.float32,)
_F8 = (torch.float8_e4m3fn,)
_ROWS = {**_FLOATS, torch.float8_e4m3fn: MOE_F8}
_INT = 1 << 31
_Tensor = torch.Tensor
# looked up once, since attribute by attribute is host time of every call; a torch without
# GPU support has neither, and no tensor that a call would take
_device, _raw_stream = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _need(ok, where, detail):
    if not ok:
        raise MoertError(MOE_EINVAL, where, detail)


def _check_tensor(where, name, t, dims, dtypes, shape=None, contiguous=False):
    """Checks one argument; `shape` entries of None are free."""
    _need(isinstance(t, torch.Tensor), where, f"{name} must be a tensor")
    _need(t.dim() == dims, where, f"{name} must have {dims} dimensions, has {t.dim()}")
    _need(t.dtype in dtypes, where, f"{name}: dtype {t.dtype} is not one of {', '.join(map(str, dtypes))}")
    if shape is not None:
        _need(all(w is None or w == h for w, h in zip(shape, t.shape)), where,
              f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if contiguous:
        _need(t.is_contiguous(), where, f"{name} must be contiguous")
    else:
        _need(t.numel() == 0 or t.shape[-1] == 1 or t.stride(-1) == 1, where,
              f"{name}: the elements of a row must be contiguous")
    _need(max(t.shape, default=0) < _INT, where, f"{name} is too large")


def _matrix(where, name, t, dtypes):
    """(rows, columns, elements from row to row) of a matrix with contiguous rows."""
    if t.__class__ is _Tensor and t.dtype in dtypes and t.is_contiguous():
        shape = t.shape
        if len(shape) == 2:
            R, C = shape
            if R < _INT and C < _INT:
                return R, C, C
    _check_tensor(where, name, t, 2, dtypes)
    R, C = t.shape
    return R, C, t.stride(0) if R > 1 else C + -C % 8  # a single row has no next one


def _whole(where, name, t, dtypes, shape):
    """Checks a contiguous argument of this shape."""
    if t.__class__ is _Tensor and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return
    _check_tensor(where, name, t, len(shape), dtypes, shape, True)


def _call(where, fn, tensors, stream, *args):
    """fn(*args, stream) with the tensors' common device current."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != dev or dev < 0):
            _need(t.is_cuda, where, f"tensors must be on the GPU, not on {t.device}")
            _need(False, where, "tensors are on different devices")
    if stream is not None and not isinstance(stream, int):
        _need(stream.device.index == dev, where, f"stream of {stream.device}, tensors on cuda:{dev}")
        stream = stream.cuda_stream
    if dev == _device():
        status = fn(*args, _raw_stream(dev) if stream is None else stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(stream))
    if status != MOE_OK:
        _check(status, where)


def moe_mx_quantize(x, codes, scales, stream=None):
    """x [R, C] f32 or bf16 (rows may be strided) -> codes uint8 [R, C/2], scales uint8 [R, C/32].  No gradient."""
    me = "moe_mx_quantize"
    R, C, ld = _matrix(me, "x", x, _FLOATS)
    _need(C % 32 == 0, me, "the columns must be a multiple of 32")
    _whole(me, "codes", codes, _U8, (R, C // 2))
    _whole(me, "scales", scales, _U8, (R, C // 32))
    _call(me, lib().moe_mx_quantize, (x, codes, scales), stream, x.data_ptr(), _FLOATS[x.dtype], R, C, ld,
          codes.data_ptr(), scales.data_ptr())


def moe_mx_dequantize(codes, scales, y, stream=None):
    """codes uint8 [R, C/2], scales uint8 [R, C/32] -> y [R, C] f32 or bf16 (rows may be strided).  No gradient."""
    me = "moe_mx_dequantize"
    R, C, ld = _matrix(me, "y", y, _FLOATS)
    _need(C % 32 == 0, me, "the columns must be a multiple of 32")
    _whole(me, "codes", codes, _U8, (R, C // 2))
    _whole(me, "scales", scales, _U8, (R, C // 32))
    _call(me, lib().moe_mx_dequantize, (y, codes, scales), stream, codes.data_ptr(), scales.data_ptr(), R, C,
          y.data_ptr(), _FLOATS[y.dtype], ld)


def _rows_operand(me, x, x_scales):
    """(rows, K, dtype, ldx) of x: bf16 rows, or codes with their scales."""
    if isinstance(x, torch.Tensor) and x.dtype is torch.float8_e4m3fn:
        R, K, ld = _matrix(me, "x", x, _F8)
        _need(x_scales is not None, me, "x in 8 bits needs x_scales")
        _whole(me, "x_scales", x_scales, _F32, (R, -(-K // 128)))
        return R, K, MOE_F8, ld
    if x_scales is None:
        R, K, ld = _matrix(me, "x", x, _BF16)
        return R, K, MOE_BF16, ld
    R, C, ld = _matrix(me, "x", x, _U8)
    _need(R < 2 or ld == C, me, "x: codes must be contiguous")
    _need(C % 16 == 0, me, "K must be a multiple of 32")
    _whole(me, "x_scales", x_scales, _U8, (R, C // 16))
    return R, 2 * C, MOE_MXFP4, 2 * C


def moe_mx_gemm(x, w_codes, w_scales, y, x_scales=None, stream=None):
    """y [M, N] (f32 or bf16) = x W^T, W as codes uint8 [N, K/2] and scales uint8
    [N, K/32]; x bf16 [M, K], or codes uint8 [M, K/2] with x_scales [M, K/32].  No gradient."""
    me = "moe_mx_gemm"
    M, K, x_dtype, ldx = _rows_operand(me, x, x_scales)
    _need(K % 32 == 0, me, "K must be a multiple of 32")
    N, C, _ = _matrix(me, "w_codes", w_codes, _U8)
    _whole(me, "w_codes", w_codes, _U8, (N, K // 2))
    _whole(me, "w_scales", w_scales, _U8, (N, K // 32))
    Y, C, ldy = _matrix(me, "y", y, _FLOATS)
    if Y != M or C != N:
        _need(False, me, f"y: shape {(Y, C)}, expected {(M, N)}")
    _call(me, lib().moe_mx_gemm, (x, x_scales, w_codes, w_scales, y), stream, x.data_ptr(), x_dtype,
          _ptr(x_scales), ldx, w_codes.data_ptr(), w_scales.data_ptr(), y.data_ptr(), _FLOATS[y.dtype], ldy, M, N,
          K)


def _f8_operand(me, v, codes, scales, block_rows, name):
    """Checks one F8 conversion; (matrices, rows, columns, elements from row to row, from matrix to matrix) of v."""
    if block_rows != 1 and block_rows != 128:
        _need(False, me, "block_rows must be 1 or 128")
    n, stride = 1, 0
    if block_rows == 128 and isinstance(v, torch.Tensor) and v.dim() == 3:
        if not (v.is_contiguous() and v.dtype in _FLOATS):
            _check_tensor(me, name, v, 3, _FLOATS)
        n, R, C = v.shape
        ld, stride = v.stride(1) if R > 1 else C, v.stride(0) if n > 1 else 0
        _need(n < _INT and R < _INT and C < _INT, me, f"{name} is too large")
    else:
        R, C, ld = _matrix(me, name, v, _FLOATS)
    if C % 16:
        _need(False, me, "the columns must be a multiple of 16")
    rows = R if block_rows == 1 else -(-R // 128)
    lead = () if v.dim() == 2 else (n,)
    _whole(me, "codes", codes, _F8, (*lead, R, C))
    _whole(me, "scales", scales, _F32, (*lead, rows, -(-C // 128)))
    return n, R, C, ld, stride


def moe_f8_quantize(x, codes, scales, block_rows=1, stream=None):
    """x [R, C] f32 or bf16 (rows may be strided) -> codes float8_e4m3fn [R, C],
    scales f32 [R, ceil(C/128)]; with block_rows=128 one scale per 128 x 128
    tile, [ceil(R/128), ceil(C/128)], and x may be [n, R, C] (codes and scales
    then too).  No gradient."""
    me = "moe_f8_quantize"
    n, R, C, ld, stride = _f8_operand(me, x, codes, scales, block_rows, "x")
    _call(me, lib().moe_f8_quantize, (x, codes, scales), stream, x.data_ptr(), _FLOATS[x.dtype], n, R, C, ld, stride,
          block_rows, codes.data_ptr(), scales.data_ptr())


def moe_f8_dequantize(codes, scales, y, block_rows=1, stream=None):
    """codes and scales as moe_f8_quantize leaves them -> y f32 or bf16 of the
    codes' shape (rows may be strided).  No gradient."""
    me = "moe_f8_dequantize"
    n, R, C, ld, stride = _f8_operand(me, y, codes, scales, block_rows, "y")
    _call(me, lib().moe_f8_dequantize, (y, codes, scales), stream, codes.data_ptr(), scales.data_ptr(), n, R, C,
          block_rows, y.data_ptr(), _FLOATS[y.dtype], ld, stride)


def moe_f8_gemm(x, x_scales, w, w_scales, y, stream=None):
    """y [M, N] (f32 or bf16) = x W^T; x float8_e4m3fn [M, K] (rows may be strided)
    with x_scales f32 [M, ceil(K/128)], W float8_e4m3fn [N, K] with w_scales f32
    [ceil(N/128), ceil(K/128)].  No gradient."""
    me = "moe_f8_gemm"
    M, K, ldx = _matrix(me, "x", x, _F8)
    KB = -(-K // 128)
    _whole(me, "x_scales", x_scales, _F32, (M, KB))
    N, C, ldw = _matrix(me, "w", w, _F8)
    if C != K or ldw != K:
        _whole(me, "w", w, _F8, (N, K))
    _whole(me, "w_scales", w_scales, _F32, (-(-N // 128), KB))
    Y, C, ldy = _matrix(me, "y", y, _FLOATS)
    if Y != M or C != N:
        _need(False, me, f"y: shape {(Y, C)}, expected {(M, N)}")
    _call(me, lib().moe_f8_gemm, (x, x_scales, w, w_scales, y), stream, x.data_ptr(), x_scales.data_ptr(), ldx,
          w.data_ptr(), w_scales.data_ptr(), y.data_ptr(), _FLOATS[y.dtype], ldy, M, N, K)


def moe_group_workspace(T, k, E):
    return lib().moe_group_workspace(T, k, E)


def moe_group_pairs(ids, n_experts, offsets, perm, workspace=None, stream=None):
    """ids int32 [T, k] -> offsets int32 [E+1], perm int32 [T*k]; workspace: any
    contiguous tensor of at least moe_group_workspace(T, k, E) bytes."""
    me = "moe_group_pairs"
    T, k, ld = _matrix(me, "ids", ids, _I32)
    _need(T < 2 or ld == k, me, "ids must be contiguous")
    _whole(me, "offsets", offsets, _I32, (n_experts + 1,))
    _whole(me, "perm", perm, _I32, (T * k,))
    nbytes = 0
    if workspace is not None:
        _need(isinstance(workspace, torch.Tensor) and workspace.is_contiguous(), me, "workspace must be a contiguous tensor")
        nbytes = workspace.numel() * workspace.element_size()
    _call(me, lib().moe_group_pairs, (ids, offsets, perm, workspace), stream, ids.data_ptr(), T, k, n_experts,
          offsets.data_ptr(), perm.data_ptr(), _ptr(workspace), nbytes)


def moe_grouped_gemm(x, w, offsets, y, x_scales=None, w_scales=None, x_index=None, x_index_div=1,
                     y_index=None, glu=False, stream=None):
    """Row p of the positions offsets[e] <= p < offsets[e+1] times expert e's W^T.
    x bf16 [n_x, K] or codes [n_x, K/2] with x_scales; w bf16 [E, N, K] or codes
    [E, N, K/2] with w_scales [E, N, K/32] (any stride from expert to expert); or
    both float8_e4m3fn, x [n_x, K] with x_scales f32 [n_x, ceil(K/128)], w [E, N, K]
    with w_scales f32 [E, ceil(N/128), ceil(K/128)] (with glu [E, 2*ceil(N/2/128),
    ceil(K/128)]: gate and up are matrices of their own); y [n_y, N], or [n_y, N/2] with glu; x_index, y_index int32 [n_rows].  The
    positions are those of an index, else the rows of x.  No gradient."""
    me = "moe_grouped_gemm"
    n_x, K, x_dtype, ldx = _rows_operand(me, x, x_scales)
    f8 = x_dtype == MOE_F8
    row, dtypes = (K, _F8) if f8 else (K, _BF16) if w_scales is None else (K // 2, _U8)
    if not (w.__class__ is torch.Tensor and w.is_contiguous() and w.dtype in dtypes and len(w.shape) == 3
            and w.shape[2] == row and max(w.shape) < _INT):
        _check_tensor(me, "w", w, 3, dtypes, (None, None, row))
        _need(w.shape[1] == 1 or w.stride(1) == row, me, "w: rows of one expert must be contiguous")
    E, N = w.shape[:2]
    ws_ptr, ws_stride = None, 0
    if f8:
        shape = (E, 2 * -(-(N // 2) // 128) if glu else -(-N // 128), -(-K // 128))
        if not (w_scales.__class__ is torch.Tensor and w_scales.is_contiguous() and w_scales.dtype in _F32
                and w_scales.shape == shape):
            _check_tensor(me, "w_scales", w_scales, 3, _F32, shape)
            _need(shape[1] == 1 or w_scales.stride(1) == shape[2], me, "w_scales: rows of one expert must be contiguous")
        ws_ptr = w_scales.data_ptr()
        ws_stride = w_scales.stride(0) * 4 if E > 1 else 0
    elif w_scales is not None:
        _need(K % 32 == 0, me, "K must be a multiple of 32")
        if not (w_scales.__class__ is torch.Tensor and w_scales.is_contiguous() and w_scales.dtype in _U8
                and w_scales.shape == (E, N, K // 32)):
            _check_tensor(me, "w_scales", w_scales, 3, _U8, (E, N, K // 32))
            _need(N == 1 or w_scales.stride(1) == K // 32, me, "w_scales: rows of one expert must be contiguous")
        ws_ptr = w_scales.data_ptr()
        ws_stride = w_scales.stride(0) if E > 1 else 0
    _whole(me, "offsets", offsets, _I32, (E + 1,))
    n_rows = n_x
    if x_index is not None or y_index is not None:
        index = y_index if x_index is None else x_index
        _check_tensor(me, "x_index" if index is x_index else "y_index", index, 1, _I32, None, True)
        n_rows = index.shape[0]
        if y_index is not None and y_index is not index:
            _whole(me, "y_index", y_index, _I32, (n_rows,))
    _need(0 < x_index_div < _INT, me, "x_index_div must be >= 1")
    n_y, cols, ldy = _matrix(me, "y", y, _FLOATS)
    if cols != (N // 2 if glu else N):
        _need(False, me, f"y has {cols} columns, expected {N // 2 if glu else N}")
    a = GroupedArgs(E, n_rows, N, K, x_dtype, MOE_F8 if f8 else MOE_BF16 if w_scales is None else MOE_MXFP4, _FLOATS[y.dtype],
                    1 if glu else 0, x.data_ptr(), _ptr(x_scales), ldx, n_x, x_index_div, _ptr(x_index),
                    w.data_ptr(), ws_ptr, w.stride(0) * w.element_size() if E > 1 else 0, ws_stride,
                    offsets.data_ptr(), y.data_ptr(), ldy, n_y, 0, _ptr(y_index))
    _call(me, lib().moe_grouped_gemm, (x, x_scales, w, w_scales, offsets, y, x_index, y_index), stream,
          ctypes.byref(a))


def moe_combine_pairs(p, w, y, ids=None, n_experts=0, stream=None):
    """y [T, H] = sum over j of w[t, j] * p[t*k + j]; p [T*k, H], w f32 [T, k];
    with ids int32 [T, k], pairs outside 0..n_experts-1 are left out.  No gradient."""
    me = "moe_combine_pairs"
    T, k, ld = _matrix(me, "w", w, _F32)
    _need(T < 2 or ld == k, me, "w must be contiguous")
    R, H, ldp = _matrix(me, "p", p, _FLOATS)
    Y, C, ldy = _matrix(me, "y", y, _FLOATS)
    if R != T * k or Y != T or C != H:
        _need(False, me, f"w {(T, k)}, p {(R, H)} and y {(Y, C)} do not belong together")
    if ids is not None:
        _whole(me, "ids", ids, _I32, (T, k))
        _need(0 < n_experts < _INT, me, "ids need n_experts >= 1")
    else:
        n_experts = 0
    _call(me, lib().moe_combine_pairs, (p, w, y, ids), stream, p.data_ptr(), _FLOATS[p.dtype], ldp, w.data_ptr(),
          _ptr(ids), n_experts, T, k, H, y.data_ptr(), _FLOATS[y.dtype], ldy)


def _norm_output(me, y, y_scales, T, H):
    """(dtype, elements from row to row) of rows that leave a norm."""
    Y, C, ldy = _matrix(me, "y", y, _ROWS)
    if Y != T or C != H:
        _need(False, me, f"y: shape {(Y, C)}, expected {(T, H)}")
    dtype = _ROWS[y.dtype]
    if dtype == MOE_F8:
        if y_scales is None:
            _need(False, me, "y in 8 bits needs y_scales")
        _whole(me, "y_scales", y_scales, _F32, (T, -(-H // 128)))
    elif y_scales is not None:
        _need(False, me, "y_scales belong to a y in 8 bits")
    return dtype, ldy


def moe_norm(x, weight, y, y_scales=None, eps=1e-6, stream=None):
    """y [T, H] = x / sqrt(mean(x^2) + eps) * weight; x f32 or bf16 [T, H], weight
    f32 or bf16 [H]; y f32, bf16, or float8_e4m3fn with y_scales f32 [T,
    ceil(H/128)].  Rows of x and y may be strided.  No gradient."""
    me = "moe_norm"
    T, H, ldx = _matrix(me, "x", x, _FLOATS)
    _whole(me, "weight", weight, _FLOATS, (H,))
    y_dtype, ldy = _norm_output(me, y, y_scales, T, H)
    _call(me, lib().moe_norm, (x, weight, y, y_scales), stream, x.data_ptr(), _FLOATS[x.dtype], ldx, weight.data_ptr(),
          _FLOATS[weight.dtype], eps, T, H, y.data_ptr(), y_dtype, None if y_scales is None else y_scales.data_ptr(), ldy)


# CombineNormArgs as bytes: a fifth of the time that its constructor takes
_COMBINE_NORM = struct.Struct("=10Q6q12i2f")


def moe_combine_norm(p, w, residual, out, ids=None, n_experts=0, post_weight=None, gate=None, scale=1.0, weight=None,
                     y=None, y_scales=None, eps=1e-6, stream=None):
    """The end of a block and the next block's norm, in fp32:
        b = sum over j of w[t, j] * p[t*k + j]       (w None: b = p)
        n = b / sqrt(mean(b^2) + eps) * post_weight  (post_weight None: n = b)
        out = r = residual + scale * gate * n
        y = r / sqrt(mean(r^2) + eps) * weight       (weight and y None: not made)
    p [T*k, H], residual and out [T, H] (out may be residual, or p where k is 1), gate [T or 1, H
    or 1], all f32 or bf16 with rows that may be strided; w f32 [T, k];
    post_weight, weight f32 or bf16 [H]; with ids int32 [T, k], pairs outside
    0..n_experts-1 are left out; y and y_scales as in moe_norm.  No gradient."""
    me = "moe_combine_norm"
    T, H, ldres = _matrix(me, "residual", residual, _FLOATS)
    R, C, ldp = _matrix(me, "p", p, _FLOATS)
    k = 1
    w_ptr = ids_ptr = post_ptr = gate_ptr = weight_ptr = y_ptr = scales_ptr = 0
    post_dtype = gate_dtype = weight_dtype = y_dtype = ldy = ldg = gate_cols = 0
    if w is not None:
        W, k, ld = _matrix(me, "w", w, _F32)
        if W != T or (T > 1 and ld != k):
            _need(False, me, "w must be contiguous, with a row per token")
        w_ptr = w.data_ptr()
    if R != T * k or C != H:
        _need(False, me, f"residual {(T, H)}, {k} rows a token and p {(R, C)} do not belong together")
    O, C, ldout = _matrix(me, "out", out, _FLOATS)
    if O != T or C != H:
        _need(False, me, f"out: shape {(O, C)}, expected {(T, H)}")
    if ids is not None:
        _whole(me, "ids", ids, _I32, (T, k))
        if not 0 < n_experts < _INT:
            _need(False, me, "ids need n_experts >= 1")
        ids_ptr = ids.data_ptr()
    else:
        n_experts = 0
    if post_weight is not None:
        _whole(me, "post_weight", post_weight, _FLOATS, (H,))
        post_ptr, post_dtype = post_weight.data_ptr(), _FLOATS[post_weight.dtype]
    if gate is not None:
        G, gate_cols, _ = _matrix(me, "gate", gate, _FLOATS)
        if G not in (1, T) or gate_cols not in (1, H):
            _need(False, me, f"gate: shape {(G, gate_cols)}, expected [1 or {T}, 1 or {H}]")
        gate_ptr, gate_dtype = gate.data_ptr(), _FLOATS[gate.dtype]
        ldg = gate.stride(0) if G > 1 else 0
    if (weight is None) != (y is None):
        _need(False, me, "weight and y belong together")
    if weight is not None:
        _whole(me, "weight", weight, _FLOATS, (H,))
        weight_ptr, weight_dtype = weight.data_ptr(), _FLOATS[weight.dtype]
        y_dtype, ldy = _norm_output(me, y, y_scales, T, H)
        y_ptr = y.data_ptr()
        if y_scales is not None:
            scales_ptr = y_scales.data_ptr()
    elif y_scales is not None:
        _need(False, me, "y_scales belong to a y in 8 bits")
    try:
        a = _COMBINE_NORM.pack(p.data_ptr(), w_ptr, ids_ptr, residual.data_ptr(), out.data_ptr(), post_ptr, gate_ptr,
                               weight_ptr, y_ptr, scales_ptr, ldp, ldres, ldout, ldg, ldy, T, k, H, n_experts, gate_cols,
                               _FLOATS[p.dtype], _FLOATS[residual.dtype], _FLOATS[out.dtype], post_dtype, gate_dtype,
                               weight_dtype, y_dtype, 0, scale, eps)
    except (struct.error, OverflowError):
        _need(False, me, f"scale {scale} or eps {eps} is no fp32 number")
    _call(me, lib().moe_combine_norm, (residual, p, out, w, ids, post_weight, gate, weight, y, y_scales), stream, a)


def moe_strerror(status: int) -> str:
    return _strerror(status)


def moe_last_error() -> str:
    return lib().moe_last_error().decode()

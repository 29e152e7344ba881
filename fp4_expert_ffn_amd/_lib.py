"""ctypes binding of libmoe.so: argument marshalling only.

Every function has the name of the C entry point it wraps and forwards to it;
device tensors are passed as ``data_ptr()`` values, the stream defaults to
torch's current HIP stream.  All arithmetic happens in the library's kernels.
A missing library is an error (there is no fallback).
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_EHIP, MOE_ENOMEM, MOE_ECACHE = range(6)
FMT = {"bf16": 0, "mxfp4": 1, "nvfp4": 2, "fp8": 3}
AMODE = {"bf16": 0, "mxfp4": 1}
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_EINVAL", 2: "MOE_EUNSUPPORTED", 3: "MOE_EHIP", 4: "MOE_ENOMEM", 5: "MOE_ECACHE"}


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class FfnArgs(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int), ("k", ctypes.c_int), ("E", ctypes.c_int), ("H", ctypes.c_int), ("I", ctypes.c_int),
        ("wfmt", ctypes.c_int), ("amode", ctypes.c_int),
        ("x", ctypes.c_void_p), ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p), ("perm", ctypes.c_void_p),
        ("slot_of_expert", ctypes.c_void_p), ("slot_pool", ctypes.c_void_p), ("slot_stride", ctypes.c_size_t),
        ("shared_blob", ctypes.c_void_p), ("expert_mask", ctypes.c_void_p),
        ("y", ctypes.c_void_p), ("topk_w", ctypes.c_void_p), ("inv", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class LayerArgs(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("renormalize", ctypes.c_int), ("topk_ids", ctypes.c_void_p),
                ("ffn", FfnArgs)]


class CacheStep(ctypes.Structure):
    _fields_ = [
        ("layer", ctypes.c_int), ("logits", ctypes.c_void_p), ("renormalize", ctypes.c_int),
        ("topk_ids", ctypes.c_void_p), ("host_counts", ctypes.c_void_p), ("host_map", ctypes.c_void_p),
        ("dev_map", ctypes.c_void_p), ("host_blobs", ctypes.c_void_p), ("ffn", FfnArgs),
        ("trace_expert", ctypes.c_void_p), ("trace_slot", ctypes.c_void_p), ("trace_hit", ctypes.c_void_p),
        ("trace_evicted", ctypes.c_void_p), ("n_experts", ctypes.c_int),
    ]


class CachePrefill(ctypes.Structure):
    _fields_ = [
        ("layer", ctypes.c_int), ("logits", ctypes.c_void_p), ("renormalize", ctypes.c_int),
        ("topk_ids", ctypes.c_void_p), ("dev_map", ctypes.c_void_p), ("ffn", FfnArgs),
        ("trace_slot", ctypes.c_void_p), ("trace_hit", ctypes.c_void_p), ("trace_evicted", ctypes.c_void_p),
    ]


class BwCalib(ctypes.Structure):
    _fields_ = [("copy_us", ctypes.c_double), ("cpu_us", ctypes.c_double), ("h2d_gbs", ctypes.c_double),
                ("host_gbs", ctypes.c_double), ("copy_ratio", ctypes.c_float)]


class Hybrid(ctypes.Structure):
    _fields_ = [("copy_ratio", ctypes.c_float), ("threads", ctypes.c_int), ("host_x", ctypes.c_void_p),
                ("host_perm", ctypes.c_void_p), ("host_offsets", ctypes.c_void_p), ("host_y", ctypes.c_void_p),
                ("cpu_experts", ctypes.c_longlong)]


class Router(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int), ("n_group", ctypes.c_int), ("topk_group", ctypes.c_int),
                ("group_rank", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float),
                ("bias", ctypes.c_void_p)]


class NormArgs(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int), ("H", ctypes.c_int), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("weight_f32", ctypes.c_int), ("eps", ctypes.c_float),
        ("residual", ctypes.c_void_p), ("residual_out", ctypes.c_void_p), ("residual_f32", ctypes.c_int),
        ("ldr", ctypes.c_int64), ("out", ctypes.c_void_p), ("ldo", ctypes.c_int64), ("qmode", ctypes.c_int),
        ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("q_scale", ctypes.c_void_p),
    ]


class LinearArgs(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int), ("qmode", ctypes.c_int),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_scale", ctypes.c_void_p),
        ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64), ("w_scale", ctypes.c_void_p),
        ("bias", ctypes.c_void_p), ("fn", ctypes.c_int), ("gated", ctypes.c_int),
        ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
        ("out", ctypes.c_void_p), ("out_f32", ctypes.c_int), ("ldo", ctypes.c_int64),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
    ]


class ExpertCanonical(ctypes.Structure):
    _fields_ = [
        ("fmt", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
        ("gate_q", ctypes.c_void_p), ("gate_s", ctypes.c_void_p), ("gate_g", ctypes.c_float),
        ("up_q", ctypes.c_void_p), ("up_s", ctypes.c_void_p), ("up_g", ctypes.c_float),
        ("down_q", ctypes.c_void_p), ("down_s", ctypes.c_void_p), ("down_g", ctypes.c_float),
    ]


SCORE = {"softmax": 0, "sigmoid": 1}
GROUP_RANK = {"max": 0, "top2": 1}
FN = {"none": 0, "silu": 1, "gelu_tanh": 2, "gelu_erf": 3, "relu": 4}
QMODE = {"none": 0, "fp8": 1, "mxfp8": 2}

# name -> (restype, argtypes); the exported C ABI (include/moe.h)
_vp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_i64 = ctypes.c_int64
SIGNATURES = {
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_version": (ctypes.c_char_p, []),
    "moe_router_logits": (_i, [_vp, _vp, _i, _i, _i, _vp, _vp]),
    "moe_route": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp]),
    "moe_permute": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "moe_route_permute": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_route_scored": (_i, [ctypes.POINTER(Router), _vp, _i, _i, _i, _vp, _vp, _vp]),
    "moe_route_scored_permute": (_i, [ctypes.POINTER(Router), _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_blob_bytes": (_sz, [_i, _i, _i]),
    "moe_prepack_expert": (_i, [ctypes.POINTER(ExpertCanonical), _vp, _sz]),
    "moe_expert_ffn_workspace_size": (_sz, [ctypes.POINTER(FfnArgs)]),
    "moe_expert_ffn": (_i, [ctypes.POINTER(FfnArgs), _vp]),
    "moe_expert_ffn_noalloc": (_i, [ctypes.POINTER(FfnArgs), _vp]),
    "moe_layer": (_i, [ctypes.POINTER(LayerArgs), _vp]),
    "moe_layer_traced": (_i, [ctypes.POINTER(LayerArgs), _vp, _vp, _i, _vp]),
    "moe_expert_ffn_traced": (_i, [ctypes.POINTER(FfnArgs), _vp, _vp, _i, _vp]),
    "moe_combine": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp]),
    "moe_quantize_mxfp4": (_i, [_vp, _i, _i, _vp, _vp, _vp]),
    "moe_rmsnorm": (_i, [ctypes.POINTER(NormArgs), _vp]),
    "moe_quantize_fp8": (_i, [_vp, _i64, _i, _i, _i, _vp, _vp, _vp]),
    "moe_linear_workspace_size": (_sz, [ctypes.POINTER(LinearArgs)]),
    "moe_linear": (_i, [ctypes.POINTER(LinearArgs), _vp]),
    "moe_dequant_blob": (_i, [_vp, _i, _vp, _vp]),
    "moe_debug_fp4_codes": (_i, [ctypes.POINTER(FfnArgs), _i, _vp, _vp, _vp]),
    "moe_cache_create": (_vp, [_i, _sz, _vp, _i, _i]),
    "moe_cache_destroy": (None, [_vp]),
    "cache_lookup": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp]),
    "cache_fill": (_i, [_vp, _i, _i, _i, _vp, _vp, _vp]),
    "moe_cache_mark_used": (_i, [_vp, _vp, _i, _vp]),
    "moe_cache_reset": (_i, [_vp]),
    "moe_cache_use_copy_engine": (_i, [_vp, _i]),
    "moe_cache_use_router": (_i, [_vp, _i, ctypes.POINTER(Router)]),
    "moe_cache_pin_resident": (_i, [_vp, _i, _i]),
    "moe_cache_stats": (_i, [_vp, _vp, _vp, _vp]),
    "moe_cache_map_bytes": (_sz, [_i]),
    "moe_cache_decode_step": (_i, [_vp, ctypes.POINTER(CacheStep), _vp, _vp]),
    "moe_cache_resize": (_i, [_vp, _i, _vp, _vp]),
    "moe_cache_prefetch_layer": (_i, [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_cache_prefill_step": (_i, [_vp, ctypes.POINTER(CachePrefill), _vp]),
    "moe_cpu_expert_ffn": (_i, [_vp, _vp, _i, _vp, _i]),
    "moe_calibrate_bw": (_i, [_vp, _vp, _i, _i, _vp, ctypes.POINTER(BwCalib)]),
    "moe_cache_decode_step_hybrid": (_i, [_vp, ctypes.POINTER(CacheStep), ctypes.POINTER(Hybrid), _vp, _vp]),
}

_lib = None


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(python -m fp4_expert_ffn_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(st: int, what: str):
    if st != MOE_OK:
        raise MoeError(st, f"{what}: {lib().moe_last_error().decode()}")


def ptr(t) -> int | None:
    """Device/host address of a torch tensor, numpy array, int or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def stream_handle(stream=None) -> int | None:
    if stream is None:
        import torch
        # the handle alone: the Stream object of torch.cuda.current_stream() costs 2.7 us a call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def moe_last_error() -> str:
    return lib().moe_last_error().decode()


def moe_version() -> str:
    return lib().moe_version().decode()


def moe_router_logits(x, w_router, T, H, E, logits, stream=None):
    _check(lib().moe_router_logits(ptr(x), ptr(w_router), T, H, E, ptr(logits), stream_handle(stream)),
           "moe_router_logits")


def moe_route(logits, T, E, k, renormalize, topk_ids, topk_w, stream=None):
    _check(lib().moe_route(ptr(logits), T, E, k, int(renormalize), ptr(topk_ids), ptr(topk_w), stream_handle(stream)),
           "moe_route")


def moe_permute(topk_ids, T, k, E, counts, offsets, perm, inv, stream=None):
    _check(lib().moe_permute(ptr(topk_ids), T, k, E, ptr(counts), ptr(offsets), ptr(perm), ptr(inv),
                             stream_handle(stream)), "moe_permute")


def moe_route_permute(logits, T, E, k, renormalize, topk_ids, topk_w, counts, offsets, perm, inv, stream=None):
    _check(lib().moe_route_permute(ptr(logits), T, E, k, int(renormalize), ptr(topk_ids), ptr(topk_w), ptr(counts),
                                   ptr(offsets), ptr(perm), ptr(inv), stream_handle(stream)), "moe_route_permute")


def moe_blob_bytes(fmt, H, I) -> int:
    return int(lib().moe_blob_bytes(FMT.get(fmt, fmt), H, I))


def moe_prepack_expert(fmt, H, I, gate, up, down) -> np.ndarray:
    """gate/up/down: (codes_or_bf16, scales_or_None, g) numpy arrays in canonical layout.

    Returns the blob as a host uint8 array."""
    f = FMT.get(fmt, fmt)
    keep = []

    def arr(a):
        if a is None:
            return None
        a = np.ascontiguousarray(a)
        keep.append(a)
        return a.ctypes.data

    c = ExpertCanonical(f, H, I,
                        arr(gate[0]), arr(gate[1]), float(gate[2]),
                        arr(up[0]), arr(up[1]), float(up[2]),
                        arr(down[0]), arr(down[1]), float(down[2]))
    n = moe_blob_bytes(f, H, I)
    out = np.empty(max(n, 1), np.uint8)
    _check(lib().moe_prepack_expert(ctypes.byref(c), out.ctypes.data, n), "moe_prepack_expert")
    return out


def ffn_args(**kw) -> FfnArgs:
    a = FfnArgs()
    for name, _ in FfnArgs._fields_:
        if name in kw:
            v = kw.pop(name)
            if name == "wfmt":
                v = FMT.get(v, v)
            elif name == "amode":
                v = AMODE.get(v, v)
            elif name in ("T", "k", "E", "H", "I", "slot_stride", "workspace_bytes"):
                v = int(v)
            else:
                v = ptr(v)
            setattr(a, name, v)
    if kw:
        raise TypeError(f"unknown moe_ffn_args fields: {sorted(kw)}")
    return a


def moe_expert_ffn_workspace_size(args: FfnArgs) -> int:
    return int(lib().moe_expert_ffn_workspace_size(ctypes.byref(args)))


def moe_expert_ffn(args: FfnArgs, stream=None):
    _check(lib().moe_expert_ffn(ctypes.byref(args), stream_handle(stream)), "moe_expert_ffn")


def moe_layer(args: LayerArgs, stream=None):
    """Routing, expert FFN and combine of one layer call (args.ffn.out required)."""
    _check(lib().moe_layer(ctypes.byref(args), stream_handle(stream)), "moe_layer")


def moe_layer_traced(args: LayerArgs, events, stream=None) -> int:
    arr = (ctypes.c_void_p * max(len(events), 1))(*[e.cuda_event for e in events])
    n = ctypes.c_int(0)
    _check(lib().moe_layer_traced(ctypes.byref(args), stream_handle(stream), arr, len(events), ctypes.byref(n)),
           "moe_layer_traced")
    return n.value


def moe_expert_ffn_noalloc(args: FfnArgs, stream=None):
    """moe_expert_ffn on the library's static device scratch (args.workspace is ignored)."""
    _check(lib().moe_expert_ffn_noalloc(ctypes.byref(args), stream_handle(stream)), "moe_expert_ffn_noalloc")


def moe_expert_ffn_traced(args: FfnArgs, events, stream=None) -> int:
    """moe_expert_ffn recording the given events (torch.cuda.Event, already
    created) around its kernel launches; returns how many were recorded."""
    arr = (ctypes.c_void_p * max(len(events), 1))(*[e.cuda_event for e in events])
    n = ctypes.c_int(0)
    _check(lib().moe_expert_ffn_traced(ctypes.byref(args), stream_handle(stream), arr, len(events), ctypes.byref(n)),
           "moe_expert_ffn_traced")
    return n.value


def moe_combine(y, inv, topk_w, y_shared, T, k, H, out, stream=None):
    _check(lib().moe_combine(ptr(y), ptr(inv), ptr(topk_w), ptr(y_shared), T, k, H, ptr(out), stream_handle(stream)),
           "moe_combine")


def moe_quantize_mxfp4(x, rows, cols, q, s, stream=None):
    _check(lib().moe_quantize_mxfp4(ptr(x), rows, cols, ptr(q), ptr(s), stream_handle(stream)), "moe_quantize_mxfp4")


def moe_debug_fp4_codes(args: FfnArgs, which, q, s, stream=None):
    _check(lib().moe_debug_fp4_codes(ctypes.byref(args), int(which), ptr(q), ptr(s), stream_handle(stream)),
           "moe_debug_fp4_codes")


# ------------------------------------------------------------ tensor arguments
# The argument builders below take torch tensors (checked: type, shape, row
# stride, device) or raw addresses (unchecked, with the sizes given).

_BF16 = ("bfloat16", "int16", "uint16")
_E4M3 = ("float8_e4m3fn", "uint8")
_E8M0 = ("float8_e8m0fnu", "uint8")
_F32 = ("float32",)


_NAMES = {}  # dtype -> its name: DenseLayer.forward checks some 20 tensors a call, and making the name anew costs 0.5 us


def _type_name(dtype) -> str:
    n = _NAMES.get(dtype)
    if n is None:
        n = _NAMES[dtype] = str(dtype).replace("torch.", "")
    return n


def _bad(what: str):
    raise MoeError(MOE_EINVAL, what)


class _Taken:
    """Collects the tensors of one argument struct: the device they share, and references that keep them alive."""

    def __init__(self, who: str):
        self.who, self.device, self.keep = who, None, []

    def __call__(self, name, t, dtypes, shape):
        """Address of tensor `t` (None and ints pass) after checking it against the names of its
        possible types and its shape; the last dimension must be dense."""
        if t is None or isinstance(t, int):
            return t
        if _type_name(t.dtype) not in dtypes:
            _bad(f"{self.who}: {name} is {t.dtype}, expected {' or '.join(dtypes)}")
        if t.shape != shape:
            _bad(f"{self.who}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        d = t.get_device()
        if d < 0:
            _bad(f"{self.who}: {name} is on {t.device}, not on a GPU")
        if self.device is None:
            self.device = d
        elif d != self.device:
            _bad(f"{self.who}: {name} is on {t.device}, other arguments on cuda:{self.device}")
        self.keep.append(t)
        return t.data_ptr()

    def dense(self, name, t, dtypes, shape):
        if t is not None and not isinstance(t, int) and not t.is_contiguous():
            _bad(f"{self.who}: {name} is not contiguous")
        return self(name, t, dtypes, shape)

    def rows(self, name, t, dtypes, shape):
        """(address, row stride in elements) of a [rows, cols] tensor with dense rows."""
        p = self(name, t, dtypes, shape)
        if t is None or isinstance(t, int):
            return p, 0
        if t.is_contiguous():
            return p, 0 if shape[0] <= 1 else shape[1]
        if shape[1] > 1 and t.stride(1) != 1:
            _bad(f"{self.who}: the rows of {name} are not dense (strides {tuple(t.stride())})")
        if shape[0] <= 1:
            return p, 0
        if t.stride(0) < shape[1]:
            _bad(f"{self.who}: the rows of {name} overlap (strides {tuple(t.stride())})")
        return p, t.stride(0)

    def done(self, a):
        a._keep, a._device = self.keep, self.device
        return a


def _current(a, what: str):
    """The call's tensors must lie on the current device (its stream runs the kernels)."""
    d = a.device if isinstance(a, _Taken) else getattr(a, "_device", None)
    if d is not None:
        import torch
        if torch.cuda.current_device() != d:
            _bad(f"{what}: tensors on cuda:{d}, current device cuda:{torch.cuda.current_device()}")


def _is_f32(t, flag):
    return int(flag) if t is None or isinstance(t, int) else int(_type_name(t.dtype) == "float32")


def norm_args(*, x, weight=None, eps=1e-6, residual=None, residual_out=None, out=None, q=None, q_scale=None,
              qmode="none", T=None, H=None, weight_f32=False, residual_f32=False) -> NormArgs:
    """Arguments of moe_rmsnorm: x [T,H] bf16; weight [H] and residual [T,H] bf16 or fp32 (taken from
    the tensors; the flags are for raw addresses); residual_out like residual; out [T,H] bf16; q [T,H]
    E4M3 codes with q_scale fp32 [T] (qmode "fp8") or E8M0 [H/128, T, 4] (qmode "mxfp8")."""
    t = _Taken("norm_args")
    if not isinstance(x, int):
        if x.dim() != 2:
            _bad(f"norm_args: x has shape {tuple(x.shape)}, expected [T, H]")
        T, H = x.shape
    a = NormArgs()
    a.T, a.H, a.eps, a.qmode = int(T), int(H), float(eps), QMODE.get(qmode, qmode)
    a.x, a.ldx = t.rows("x", x, _BF16, (T, H))
    a.weight, a.weight_f32 = t.dense("weight", weight, _BF16 + _F32, (H,)), _is_f32(weight, weight_f32)
    a.residual_f32 = _is_f32(residual, residual_f32)
    rtypes = _F32 if a.residual_f32 else _BF16
    a.residual, a.ldr = t.rows("residual", residual, rtypes, (T, H))
    a.residual_out, ldro = t.rows("residual_out", residual_out, rtypes, (T, H))
    if ldro != a.ldr and residual_out is not None and not isinstance(residual_out, int):
        _bad("norm_args: residual and residual_out have different row strides")
    a.out, a.ldo = t.rows("out", out, _BF16, (T, H))
    a.q, a.ldq = t.rows("q", q, _E4M3, (T, H))
    if a.qmode == QMODE["mxfp8"]:
        a.q_scale = t.dense("q_scale", q_scale, _E8M0, (H // 128, T, 4))
    else:
        a.q_scale = t.dense("q_scale", q_scale, _F32, (T,))
    return t.done(a)


def router(*, score="softmax", n_group=1, topk_group=1, group_rank="max", renormalize=True, scale=1.0,
           bias=None) -> Router:
    """A router for moe_route_scored: score "softmax" or "sigmoid", n_group groups of which the topk_group best
    by group_rank ("max" or "top2") are kept, bias [E] fp32 (device) for the choice alone."""
    t = _Taken("router")
    r = Router()
    r.score, r.group_rank = SCORE.get(score, score), GROUP_RANK.get(group_rank, group_rank)
    r.n_group, r.topk_group, r.renormalize, r.scale = int(n_group), int(topk_group), int(renormalize), float(scale)
    r._experts = None if bias is None or isinstance(bias, int) else bias.numel()
    r.bias = t.dense("bias", bias, _F32, (r._experts,))
    return t.done(r)


def _check_route(what: str, r: Router, E: int, floats, ints):
    """The router's bias fits E; floats (fp32) and ints (int32), pairs of a tensor and its least length, are
    dense and on the current device.  A decode step's routing takes 7 us: no names or strings before a fault."""
    import torch
    n = getattr(r, "_experts", None)
    if n is not None and n != E:
        _bad(f"{what}: the router's bias has {n} experts, E={E}")
    dev = getattr(r, "_device", None)
    for kind, pairs in ((torch.float32, floats), (torch.int32, ints)):
        for t, need in pairs:
            if t is None or t.__class__ is int:
                continue
            d = t.get_device()
            if t.dtype is not kind or d < 0 or not t.is_contiguous() or t.numel() < need:
                _bad(f"{what}: a {t.dtype} tensor of {t.numel()} values on {t.device} where a dense {kind} GPU "
                     f"tensor of at least {need} values belongs")
            if dev is None:
                dev = d
            elif d != dev:
                _bad(f"{what}: tensors on cuda:{dev} and cuda:{d}")
    if dev is not None and torch.cuda.current_device() != dev:
        _bad(f"{what}: tensors on cuda:{dev}, current device cuda:{torch.cuda.current_device()}")


def moe_route_scored(r: Router, logits, T, E, k, topk_ids, topk_w, stream=None):
    _check_route("moe_route_scored", r, E, ((logits, T * E), (topk_w, T * k)), ((topk_ids, T * k),))
    _check(lib().moe_route_scored(ctypes.byref(r), ptr(logits), T, E, k, ptr(topk_ids), ptr(topk_w),
                                  stream_handle(stream)), "moe_route_scored")


def moe_route_scored_permute(r: Router, logits, T, E, k, topk_ids, topk_w, counts, offsets, perm, inv, stream=None):
    n = T * k
    _check_route("moe_route_scored_permute", r, E, ((logits, T * E), (topk_w, n)),
                 ((topk_ids, n), (counts, E), (offsets, E + 1), (perm, n), (inv, n)))
    _check(lib().moe_route_scored_permute(ctypes.byref(r), ptr(logits), T, E, k, ptr(topk_ids), ptr(topk_w),
                                          ptr(counts), ptr(offsets), ptr(perm), ptr(inv), stream_handle(stream)),
           "moe_route_scored_permute")


def moe_rmsnorm(args: NormArgs, stream=None):
    _current(args, "moe_rmsnorm")
    _check(lib().moe_rmsnorm(ctypes.byref(args), stream_handle(stream)), "moe_rmsnorm")


def moe_quantize_fp8(x, rows, cols, qmode, q, q_scale, stream=None, ldx=0):
    """8-bit rows of bf16 x [rows, cols] (tensor: its own row stride; raw address: ldx elements, 0 dense):
    dense E4M3 codes q [rows, cols], q_scale fp32 [rows] (qmode "fp8") or E8M0 [cols/128, rows, 4] ("mxfp8")."""
    t, qm = _Taken("moe_quantize_fp8"), QMODE.get(qmode, qmode)
    xp, ld = t.rows("x", x, _BF16, (rows, cols))
    qp = t.dense("q", q, _E4M3, (rows, cols))
    sp = (t.dense("q_scale", q_scale, _E8M0, (cols // 128, rows, 4)) if qm == QMODE["mxfp8"] else
          t.dense("q_scale", q_scale, _F32, (rows,)))
    _current(t, "moe_quantize_fp8")
    _check(lib().moe_quantize_fp8(xp, ld or ldx, rows, cols, qm, qp, sp, stream_handle(stream)), "moe_quantize_fp8")


def linear_args(*, x, w, out, fmt="bf16", x_scale=None, w_scale=None, bias=None, act="none", gated=False,
                residual=None, T=None, N=None, K=None, out_f32=False) -> LinearArgs:
    """Arguments of moe_linear (workspace left empty): x [T,K] and w [R,K] bf16 (fmt "bf16") or E4M3 codes with
    x_scale / w_scale (fmt "fp8": fp32 [T] / [R]; "mxfp8": E8M0 [K/128, T, 4] / [K/128, R, 4]); R = N, gated 2 N;
    bias fp32 [R]; residual [T,N] bf16; out [T,N] bf16 or fp32."""
    t = _Taken("linear_args")
    for name, v in (("x", x), ("w", w), ("out", out)):
        if not isinstance(v, int) and v.dim() != 2:
            _bad(f"linear_args: {name} has shape {tuple(v.shape)}, expected two dimensions")
    if not isinstance(x, int):
        T, K = x.shape
    if not isinstance(out, int):
        N = out.shape[1]
    R = 2 * N if gated else N
    a = LinearArgs()
    a.T, a.N, a.K, a.gated = int(T), int(N), int(K), int(gated)
    a.qmode = QMODE["none"] if fmt == "bf16" else QMODE.get(fmt, fmt)
    a.fn = FN.get(act, act)
    types = _BF16 if a.qmode == QMODE["none"] else _E4M3
    a.x, a.ldx = t.rows("x", x, types, (T, K))
    a.w, a.ldw = t.rows("w", w, types, (R, K))
    if a.qmode == QMODE["mxfp8"]:
        a.x_scale = t.dense("x_scale", x_scale, _E8M0, (K // 128, T, 4))
        a.w_scale = t.dense("w_scale", w_scale, _E8M0, (K // 128, R, 4))
    else:
        a.x_scale = t.dense("x_scale", x_scale, _F32, (T,))
        a.w_scale = t.dense("w_scale", w_scale, _F32, (R,))
    a.bias = t.dense("bias", bias, _F32, (R,))
    a.residual, a.ldr = t.rows("residual", residual, _BF16, (T, N))
    a.out_f32 = _is_f32(out, out_f32)
    a.out, a.ldo = t.rows("out", out, _F32 if a.out_f32 else _BF16, (T, N))
    return t.done(a)


def moe_linear_workspace_size(args: LinearArgs) -> int:
    return int(lib().moe_linear_workspace_size(ctypes.byref(args)))


def moe_linear(args: LinearArgs, stream=None):
    _current(args, "moe_linear")
    _check(lib().moe_linear(ctypes.byref(args), stream_handle(stream)), "moe_linear")


def moe_dequant_blob(blob, which, out, stream=None):
    _check(lib().moe_dequant_blob(ptr(blob), which, ptr(out), stream_handle(stream)), "moe_dequant_blob")


class Cache:
    """Owner of a moe_cache handle (host LRU metadata + HIP events)."""

    def __init__(self, num_slots, slot_bytes, slot_pool, num_layers, num_experts):
        h = lib().moe_cache_create(num_slots, slot_bytes, ptr(slot_pool), num_layers, num_experts)
        if not h:
            raise MoeError(MOE_EINVAL, moe_last_error())
        self.handle = h
        self.num_slots, self.num_experts = num_slots, num_experts
        self._device = slot_pool.device.index if getattr(slot_pool, "is_cuda", False) else None
        self._routers = {}  # layer (-1: every layer) -> router: their biases stay alive with the cache

    def close(self):
        if self.handle:
            lib().moe_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def moe_cache_create(num_slots, slot_bytes, slot_pool, num_layers, num_experts) -> Cache:
    return Cache(num_slots, slot_bytes, slot_pool, num_layers, num_experts)


def moe_cache_destroy(cache: Cache):
    cache.close()


def cache_lookup(cache: Cache, layer: int, ids):
    """ids: distinct ascending expert ids.  Returns (slot, hit, evicted_key) numpy arrays."""
    ids = np.ascontiguousarray(ids, dtype=np.int32)
    n = ids.size
    slot = np.empty(n, np.int32)
    hit = np.empty(n, np.uint8)
    ev = np.empty(n, np.int32)
    _check(lib().cache_lookup(cache.handle, layer, ids.ctypes.data, n, slot.ctypes.data, hit.ctypes.data,
                              ev.ctypes.data), "cache_lookup")
    return slot, hit, ev


def cache_fill(cache: Cache, layer, expert, slot, host_src, copy_stream=None, compute_stream=None):
    _check(lib().cache_fill(cache.handle, layer, expert, slot, ptr(host_src), stream_handle(copy_stream),
                            stream_handle(compute_stream)), "cache_fill")


def moe_cache_mark_used(cache: Cache, slots, stream=None):
    s = np.ascontiguousarray(slots, dtype=np.int32)
    _check(lib().moe_cache_mark_used(cache.handle, s.ctypes.data, s.size, stream_handle(stream)),
           "moe_cache_mark_used")


def moe_cache_reset(cache: Cache):
    _check(lib().moe_cache_reset(cache.handle), "moe_cache_reset")


def moe_cache_use_copy_engine(cache: Cache, on: bool):
    _check(lib().moe_cache_use_copy_engine(cache.handle, 1 if on else 0), "moe_cache_use_copy_engine")


def moe_cache_use_router(cache: Cache, layer: int, r: Router | None):
    """Steps of `layer` (-1: every layer) route by the scored router r (None: softmax top-k again).
    The bias needs the cache's number of experts and its pool's device; the cache keeps it alive until
    another router takes its place (steps still queued by then need it kept by the caller)."""
    if r is not None:
        n, dev = getattr(r, "_experts", None), getattr(r, "_device", None)
        if n is not None and n != cache.num_experts:
            _bad(f"moe_cache_use_router: the router's bias has {n} experts, the cache {cache.num_experts}")
        if dev is not None and cache._device is not None and dev != cache._device:
            _bad(f"moe_cache_use_router: the router's bias is on cuda:{dev}, the cache's pool on cuda:{cache._device}")
    _check(lib().moe_cache_use_router(cache.handle, int(layer), None if r is None else ctypes.byref(r)),
           "moe_cache_use_router")
    if layer == -1:
        cache._routers.clear()
    cache._routers[layer] = r


def moe_cache_pin_resident(cache: Cache, layer, s0):
    _check(lib().moe_cache_pin_resident(cache.handle, layer, s0), "moe_cache_pin_resident")


def moe_cache_stats(cache: Cache):
    """(hits, misses, bytes_filled) since creation or reset."""
    v = (ctypes.c_longlong * 3)()
    _check(lib().moe_cache_stats(cache.handle, ctypes.byref(v, 0), ctypes.byref(v, 8), ctypes.byref(v, 16)),
           "moe_cache_stats")
    return int(v[0]), int(v[1]), int(v[2])


def moe_cache_map_bytes(E: int) -> int:
    return int(lib().moe_cache_map_bytes(E))


def moe_cache_decode_step(cache: Cache, step: CacheStep, copy_stream=None, compute_stream=None):
    _check(lib().moe_cache_decode_step(cache.handle, ctypes.byref(step), stream_handle(copy_stream),
                                       stream_handle(compute_stream)), "moe_cache_decode_step")


def moe_cache_resize(cache: Cache, num_slots: int, slot_pool, stream=None):
    _check(lib().moe_cache_resize(cache.handle, int(num_slots), ptr(slot_pool), stream_handle(stream)),
           "moe_cache_resize")


def moe_cache_prefetch_layer(cache: Cache, layer, host_blobs, host_map, dev_map, trace=None, copy_stream=None,
                             compute_stream=None):
    """host_blobs: ctypes array of E pinned blob addresses; trace: None or
    (slot int32 [E], hit uint8 [E], evicted int32 [E]) numpy arrays."""
    t = (None, None, None) if trace is None else tuple(a.ctypes.data for a in trace)
    _check(lib().moe_cache_prefetch_layer(cache.handle, int(layer), ctypes.cast(host_blobs, ctypes.c_void_p),
                                          ptr(host_map), ptr(dev_map), *t, stream_handle(copy_stream),
                                          stream_handle(compute_stream)), "moe_cache_prefetch_layer")


def moe_cache_prefill_step(cache: Cache, step: CachePrefill, compute_stream=None):
    _check(lib().moe_cache_prefill_step(cache.handle, ctypes.byref(step), stream_handle(compute_stream)),
           "moe_cache_prefill_step")


def moe_cpu_expert_ffn(blob, x, n, y, threads=1):
    """blob, x (bf16 bits [n,H]), y (fp32 [n,H]): host arrays."""
    _check(lib().moe_cpu_expert_ffn(ptr(blob), ptr(x), int(n), ptr(y), int(threads)), "moe_cpu_expert_ffn")


def moe_calibrate_bw(host_blob, dev_buf, reps=8, threads=1, copy_stream=None) -> BwCalib:
    out = BwCalib()
    _check(lib().moe_calibrate_bw(ptr(host_blob), ptr(dev_buf), int(reps), int(threads), stream_handle(copy_stream),
                                  ctypes.byref(out)), "moe_calibrate_bw")
    return out


def moe_cache_decode_step_hybrid(cache: Cache, step: CacheStep, hybrid: Hybrid, copy_stream=None, compute_stream=None):
    _check(lib().moe_cache_decode_step_hybrid(cache.handle, ctypes.byref(step), ctypes.byref(hybrid),
                                              stream_handle(copy_stream), stream_handle(compute_stream)),
           "moe_cache_decode_step_hybrid")

"""Python binding of libmoe (include/libmoe.h): argument marshalling only.

Every function has the name of the C entry point it calls.  Tensors are torch tensors on the
GPU; calls enqueue on torch's current stream (or `stream=`) and do not synchronise.  Every step
of the MoE layer runs in libmoe's HIP kernels; this module only passes pointers and sizes.  A
missing libmoe.so is an error (build it with `python -m routed_expert_grouped_amd.build`).
"""
from __future__ import annotations

import ctypes
import os
import types

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_DEVICE = range(5)
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_W_FP8_E4M3_B128, MOE_W_BF16, MOE_W_MXFP4_G32 = 0, 1, 2
MOE_ROUTER_W_BF16, MOE_ROUTER_W_F32 = 0, 1
SCORE_FN = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}

EXPORTS = ("moe_route", "moe_permute_workspace_size", "moe_permute", "moe_expert_gate_up", "moe_expert_down",
           "moe_expert_gate_up_shared", "moe_expert_down_shared",
           "moe_expert_ffn_workspace_size", "moe_expert_ffn", "moe_combine", "moe_quantize_act",
           "moe_expert_gate_up_a8", "moe_expert_down_a8", "moe_expert_ffn_a8_workspace_size",
           "moe_expert_ffn_a8", "moe_combine_partial", "moe_route_permute",
           "moe_permute_noalloc", "moe_rmsnorm_quantize_act", "moe_router_scores_workspace_size",
           "moe_router_scores", "moe_layer_few_workspace_size", "moe_layer_few",
           "moe_linear_a8", "moe_status_string")


class MoeError(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        super().__init__(f"{call} failed: {moe_status_string(status)} ({status})")


class MoeExpertWeights(ctypes.Structure):
    """ctypes mirror of moe_expert_weights."""
    _fields_ = [("dtype", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("H", ctypes.c_int32),
                ("I", ctypes.c_int32), ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("s_gate", ctypes.c_void_p), ("s_up", ctypes.c_void_p),
                ("s_down", ctypes.c_void_p)]


_lib = None


def lib():
    """The loaded libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmoe.so not found at {LIB_PATH}; build it with "
                               "`python -m routed_expert_grouped_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int
        W = ctypes.POINTER(MoeExpertWeights)
        L.moe_route.argtypes = [P, i32, i32, i32, i32, i32, P, P, P]
        L.moe_permute_workspace_size.argtypes = [i32, i32, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_permute.argtypes = [P, i32, i32, i32, P, P, P, P, P, ctypes.c_size_t, P]
        L.moe_permute_noalloc.argtypes = [P, i32, i32, i32, P, P, P, P, P]
        L.moe_route_permute.argtypes = [P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P]
        L.moe_expert_gate_up.argtypes = [P, i32, i32, P, P, W, P, P]
        L.moe_expert_down.argtypes = [P, i32, i32, P, W, P, P]
        L.moe_expert_gate_up_shared.argtypes = [P, i32, i32, P, P, W, W, P, P]
        L.moe_expert_down_shared.argtypes = [P, i32, i32, P, W, W, P, P]
        L.moe_expert_ffn_workspace_size.argtypes = [i32, i32, W, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_expert_ffn.argtypes = [P, i32, i32, P, P, W, P, P, ctypes.c_size_t, P]
        L.moe_combine.argtypes = [P, P, P, P, i32, i32, i32, P, P]
        L.moe_combine_partial.argtypes = [P, P, P, P, i32, i32, P, i32, i32, i32, P, P]
        L.moe_quantize_act.argtypes = [P, i32, i32, P, P, i32, P]
        L.moe_expert_gate_up_a8.argtypes = [P, P, i32, i32, i32, P, P, W, P, P]
        L.moe_expert_down_a8.argtypes = [P, P, i32, i32, i32, P, W, P, P]
        L.moe_expert_ffn_a8_workspace_size.argtypes = [i32, i32, W,
                                                       ctypes.POINTER(ctypes.c_size_t)]
        L.moe_expert_ffn_a8.argtypes = [P, i32, i32, P, P, W, P, P, ctypes.c_size_t, P]
        L.moe_rmsnorm_quantize_act.argtypes = [P, P, P, i32, i32, ctypes.c_float, P, P, P, P, i32, P]
        L.moe_router_scores_workspace_size.argtypes = [i32, i32, i32,
                                                       ctypes.POINTER(ctypes.c_size_t)]
        L.moe_router_scores.argtypes = [P, i32, i32, P, i32, i32, P, P, ctypes.c_size_t, P]
        L.moe_layer_few_workspace_size.argtypes = [i32, i32, W, ctypes.POINTER(ctypes.c_size_t)]
        L.moe_layer_few.argtypes = [P, P, i32, i32, i32, i32, W, W, P, P, P, P, ctypes.c_size_t, P]
        L.moe_linear_a8.argtypes = [P, P, i32, i32, i32, i32, P, P, P, P]
        for name in EXPORTS[:-1]:
            getattr(L, name).restype = st
        L.moe_status_string.argtypes = [st]
        L.moe_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _p(t):
    """Device pointer of a tensor (None -> NULL)."""
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(call, status):
    if status != MOE_OK:
        raise MoeError(call, status)


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


WDTYPE = {"fp8": MOE_W_FP8_E4M3_B128, "bf16": MOE_W_BF16, "mxfp4": MOE_W_MXFP4_G32}


def expert_weights(ew) -> MoeExpertWeights:
    """moe_expert_weights for an object with .wdtype ("fp8", "bf16" or "mxfp4"), .gate/.up/.down
    and .s_gate/.s_up/.s_down device tensors (the arrays must outlive the calls that use it)."""
    n, I, H = ew.gate.shape
    if ew.wdtype == "mxfp4":
        H *= 2  # two codes a byte along the input dimension
    scaled = ew.wdtype != "bf16"
    return MoeExpertWeights(WDTYPE[ew.wdtype], n, H, I,
                            ew.gate.data_ptr(), ew.up.data_ptr(), ew.down.data_ptr(),
                            ew.s_gate.data_ptr() if scaled else None,
                            ew.s_up.data_ptr() if scaled else None,
                            ew.s_down.data_ptr() if scaled else None)


def expert_slice(ew, e_begin: int, e_end: int):
    """Experts e_begin .. e_end - 1 of an object accepted by expert_weights(), as views of the
    same arrays (no copy): the weights one rank holds under expert parallelism."""
    return types.SimpleNamespace(
        wdtype=ew.wdtype, gate=ew.gate[e_begin:e_end], up=ew.up[e_begin:e_end],
        down=ew.down[e_begin:e_end],
        **{n: (None if getattr(ew, n) is None else getattr(ew, n)[e_begin:e_end])
           for n in ("s_gate", "s_up", "s_down")})


def moe_route(scores, k: int, score_fn="sigmoid", renorm: int = 1, topk_ids=None, topk_w=None,
              stream=None):
    T, E = scores.shape
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=scores.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=scores.device)
    fn = SCORE_FN[score_fn] if isinstance(score_fn, str) else int(score_fn)
    _check("moe_route", lib().moe_route(_p(scores), T, E, k, fn, int(renorm), _p(topk_ids),
                                        _p(topk_w), _s(stream)))
    return topk_ids, topk_w


FUSED_ROUTE_PERMUTE_MAX = 2048  # assignments up to which moe_route_permute runs


def moe_route_permute(scores, k: int, score_fn="sigmoid", renorm: int = 1, topk_ids=None,
                      topk_w=None, counts=None, offsets=None, perm=None, inv=None, stream=None):
    """moe_route + moe_permute in one launch (T*k <= 2048); returns ids, w, counts, offsets,
    perm, inv."""
    T, E = scores.shape
    dev, i32 = scores.device, torch.int32
    topk_ids = torch.empty((T, k), dtype=i32, device=dev) if topk_ids is None else topk_ids
    topk_w = torch.empty((T, k), dtype=torch.float32, device=dev) if topk_w is None else topk_w
    counts = torch.empty(E, dtype=i32, device=dev) if counts is None else counts
    offsets = torch.empty(E + 1, dtype=i32, device=dev) if offsets is None else offsets
    perm = torch.empty(max(1, T * k), dtype=i32, device=dev) if perm is None else perm
    inv = torch.empty(max(1, T * k), dtype=i32, device=dev) if inv is None else inv
    fn = SCORE_FN[score_fn] if isinstance(score_fn, str) else int(score_fn)
    _check("moe_route_permute",
           lib().moe_route_permute(_p(scores), T, E, k, fn, int(renorm), _p(topk_ids), _p(topk_w),
                                   _p(counts), _p(offsets), _p(perm), _p(inv), _s(stream)))
    return topk_ids, topk_w, counts, offsets, perm, inv


def moe_permute_workspace_size(T: int, k: int, E: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_permute_workspace_size",
           lib().moe_permute_workspace_size(T, k, E, ctypes.byref(n)))
    return n.value


def moe_permute(topk_ids, E: int, counts=None, offsets=None, perm=None, inv=None, ws=None,
                stream=None):
    """Returns counts, offsets, perm, inv.  `ws` (uint8 device tensor) is the call's workspace;
    None allocates one of moe_permute_workspace_size bytes (the caller must keep a passed one
    untouched until the stream has run the call)."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev) if counts is None else counts
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    perm = torch.empty(T * k, dtype=torch.int32, device=dev) if perm is None else perm
    inv = torch.empty(T * k, dtype=torch.int32, device=dev) if inv is None else inv
    if ws is None:
        need = moe_permute_workspace_size(T, k, E)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _check("moe_permute", lib().moe_permute(_p(topk_ids), T, k, E, _p(counts), _p(offsets),
                                            _p(perm), _p(inv), _p(ws),
                                            0 if ws is None else ws.numel(), _s(stream)))
    return counts, offsets, perm, inv


PERMUTE_NOALLOC_MAX_BYTES = 1 << 20  # MOE_PERMUTE_NOALLOC_MAX_BYTES


def moe_permute_noalloc(topk_ids, E: int, counts, offsets, perm, inv, stream=None):
    """moe_permute with the library's static count table instead of a workspace (the caller
    passes every output buffer; nothing is allocated here or in the call)."""
    T, k = topk_ids.shape
    _check("moe_permute_noalloc",
           lib().moe_permute_noalloc(_p(topk_ids), T, k, E, _p(counts), _p(offsets), _p(perm),
                                     _p(inv), _s(stream)))
    return counts, offsets, perm, inv


def moe_expert_gate_up(x, k: int, perm, offsets, w: MoeExpertWeights, h=None, stream=None):
    T = x.shape[0]
    if h is None:
        h = torch.empty((T * k, w.I), dtype=torch.int16, device=x.device)
    _check("moe_expert_gate_up", lib().moe_expert_gate_up(
        _p(x), T, k, _p(perm), _p(offsets), ctypes.byref(w), _p(h), _s(stream)))
    return h


def moe_expert_down(h, T: int, k: int, offsets, w: MoeExpertWeights, y=None, stream=None):
    if y is None:
        y = torch.empty((T * k, w.H), dtype=torch.int16, device=h.device)
    _check("moe_expert_down", lib().moe_expert_down(
        _p(h), T, k, _p(offsets), ctypes.byref(w), _p(y), _s(stream)))
    return y


def moe_expert_gate_up_shared(x, k: int, perm, offsets, w: MoeExpertWeights, ws: MoeExpertWeights,
                              h=None, stream=None):
    """Routed gate/up over the T*k grouped rows and the shared expert's over T more rows (h has
    T*k + T rows; row T*k + t is token t's shared-expert h)."""
    T = x.shape[0]
    if h is None:
        h = torch.empty((T * k + T, w.I), dtype=torch.int16, device=x.device)
    _check("moe_expert_gate_up_shared", lib().moe_expert_gate_up_shared(
        _p(x), T, k, _p(perm), _p(offsets), ctypes.byref(w), ctypes.byref(ws), _p(h), _s(stream)))
    return h


def moe_expert_down_shared(h, T: int, k: int, offsets, w: MoeExpertWeights, ws: MoeExpertWeights,
                           y=None, stream=None):
    """Down projection of moe_expert_gate_up_shared's h: y has T*k + T rows, the shared expert's
    output from row T*k on."""
    if y is None:
        y = torch.empty((T * k + T, w.H), dtype=torch.int16, device=h.device)
    _check("moe_expert_down_shared", lib().moe_expert_down_shared(
        _p(h), T, k, _p(offsets), ctypes.byref(w), ctypes.byref(ws), _p(y), _s(stream)))
    return y


def moe_expert_ffn_workspace_size(T: int, k: int, w: MoeExpertWeights) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_expert_ffn_workspace_size",
           lib().moe_expert_ffn_workspace_size(T, k, ctypes.byref(w), ctypes.byref(n)))
    return n.value


def moe_expert_ffn(x, k: int, perm, offsets, w: MoeExpertWeights, y=None, ws=None, stream=None):
    T = x.shape[0]
    if y is None:
        y = torch.empty((T * k, w.H), dtype=torch.int16, device=x.device)
    if ws is None:
        ws = torch.empty(max(1, moe_expert_ffn_workspace_size(T, k, w)), dtype=torch.uint8,
                         device=x.device)
    _check("moe_expert_ffn", lib().moe_expert_ffn(
        _p(x), T, k, _p(perm), _p(offsets), ctypes.byref(w), _p(y), _p(ws), ws.numel(),
        _s(stream)))
    return y, ws


def moe_combine(y, inv, topk_w, shared_y, T: int, k: int, H: int, out=None, stream=None):
    if out is None:
        out = torch.empty((T, H), dtype=torch.int16, device=y.device)
    _check("moe_combine", lib().moe_combine(_p(y), _p(inv), _p(topk_w), _p(shared_y), T, k, H,
                                            _p(out), _s(stream)))
    return out


def moe_combine_partial(y, inv, topk_ids, topk_w, e_begin: int, e_end: int, shared_y, T: int,
                        k: int, H: int, out=None, stream=None):
    if out is None:
        out = torch.empty((T, H), dtype=torch.int16, device=y.device)
    _check("moe_combine_partial",
           lib().moe_combine_partial(_p(y), _p(inv), _p(topk_ids), _p(topk_w), int(e_begin),
                                     int(e_end), _p(shared_y), T, k, H, _p(out), _s(stream)))
    return out


def exp_pitch(K: int) -> int:
    """Exponent row pitch that the FP8-activation phase calls take: K/128 rounded up to 16."""
    return (K // 128 + 15) // 16 * 16


def moe_quantize_act(x, codes=None, exps=None, pitch=None, stream=None):
    """FP8 activation quantisation of bf16 bits x [rows, K]: (codes uint8 [rows, K], exps int8
    [rows, pitch]; the exponents of row r are exps[r, :K/128])."""
    rows, K = x.shape
    pitch = exp_pitch(K) if pitch is None else pitch
    if codes is None:
        codes = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    if exps is None:
        exps = torch.empty((rows, max(1, pitch)), dtype=torch.int8, device=x.device)
    _check("moe_quantize_act", lib().moe_quantize_act(_p(x), rows, K, _p(codes), _p(exps), pitch,
                                                      _s(stream)))
    return codes, exps


def moe_expert_gate_up_a8(codes, exps, k: int, perm, offsets, w: MoeExpertWeights, h=None,
                          stream=None):
    T = codes.shape[0]
    if h is None:
        h = torch.empty((T * k, w.I), dtype=torch.int16, device=codes.device)
    _check("moe_expert_gate_up_a8", lib().moe_expert_gate_up_a8(
        _p(codes), _p(exps), exps.shape[1], T, k, _p(perm), _p(offsets), ctypes.byref(w), _p(h),
        _s(stream)))
    return h


def moe_expert_down_a8(codes, exps, T: int, k: int, offsets, w: MoeExpertWeights, y=None,
                       stream=None):
    if y is None:
        y = torch.empty((T * k, w.H), dtype=torch.int16, device=codes.device)
    _check("moe_expert_down_a8", lib().moe_expert_down_a8(
        _p(codes), _p(exps), exps.shape[1], T, k, _p(offsets), ctypes.byref(w), _p(y),
        _s(stream)))
    return y


def moe_expert_ffn_a8_workspace_size(T: int, k: int, w: MoeExpertWeights) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_expert_ffn_a8_workspace_size",
           lib().moe_expert_ffn_a8_workspace_size(T, k, ctypes.byref(w), ctypes.byref(n)))
    return n.value


def moe_expert_ffn_a8(x, k: int, perm, offsets, w: MoeExpertWeights, y=None, ws=None,
                      stream=None):
    T = x.shape[0]
    if y is None:
        y = torch.empty((T * k, w.H), dtype=torch.int16, device=x.device)
    if ws is None:
        ws = torch.empty(max(1, moe_expert_ffn_a8_workspace_size(T, k, w)), dtype=torch.uint8,
                         device=x.device)
    _check("moe_expert_ffn_a8", lib().moe_expert_ffn_a8(
        _p(x), T, k, _p(perm), _p(offsets), ctypes.byref(w), _p(y), _p(ws), ws.numel(),
        _s(stream)))
    return y, ws


def _off(t, dtype, shape, index):
    """Whether a tensor is not what a call takes: raw pointers are passed on, so another layout would
    be read as this one.  (None is an argument left out.)"""
    return t is not None and (t.dtype is not dtype or t.shape != shape or t.get_device() != index
                              or not t.is_contiguous())


def _refuse(call, index, **tensors):
    """Names the argument that _off found: name=(tensor, dtype, shape)."""
    for name, (t, dtype, shape) in tensors.items():
        if _off(t, dtype, shape, index):
            raise ValueError(f"{call}: {name} must be a contiguous {dtype} tensor of shape "
                             f"{tuple(shape)} on cuda:{index}, not {t.dtype} {tuple(t.shape)} with "
                             f"strides {t.stride()} on {t.device}")
    raise AssertionError(call)


def _where(call, t, stream):
    """(device index, stream handle) of a call on tensor t: torch's current stream of t's device, or the
    caller's `stream`, which must be of that device."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{call}: the tensors must be on a GPU, not on {t.device}")
    if stream is None:
        return index, torch._C._cuda_getCurrentRawStream(index)
    if stream.device_index != index:
        raise ValueError(f"{call}: the stream is of {stream.device}, the tensors are on {t.device}")
    return index, stream.cuda_stream


def _new(t, stream, shape, dtype):
    """A buffer on t's device that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=t.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=t.device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _run(call, index, *args):
    """The C call, with the tensors' device current (it launches there)."""
    if index == torch._C._cuda_getDevice():
        status = getattr(_lib or lib(), call)(*args)
    else:
        with torch.cuda.device(index):
            status = getattr(_lib or lib(), call)(*args)
    if status != MOE_OK:
        raise MoeError(call, status)


def moe_rmsnorm_quantize_act(x, weight, residual=None, eps: float = 1e-6, normed=True,
                             quantized=True, sum_out=None, y=None, codes=None, exps=None,
                             pitch=None, stream=None):
    """RMS norm of bf16 bits x [rows, K] (+ residual, added first) with the bf16 bits `weight` [K].
    Returns (sum, y, codes, exps): the stored sum (None without a residual), the normalised rows
    (None unless `normed`) and their FP8 codes and block exponents as moe_quantize_act's (None unless
    `quantized`).  sum_out may be x or residual: the residual stream updated in place."""
    call = "moe_rmsnorm_quantize_act"
    if x.dim() != 2:
        raise ValueError(f"{call}: x must have two dimensions")
    dev, st = _where(call, x, stream)
    shape, b16 = x.shape, torch.int16
    rows, K = shape
    if quantized:
        pitch = exps.shape[1] if exps is not None else exp_pitch(K) if pitch is None else pitch
    else:
        codes = exps = None
        pitch = 0
    if not normed:
        y = None
    if residual is None and sum_out is not None:
        raise ValueError(f"{call}: sum_out needs a residual")
    u8, i8 = torch.uint8, torch.int8
    if (_off(x, b16, shape, dev) or _off(weight, b16, (K,), dev) or _off(residual, b16, shape, dev)
            or _off(sum_out, b16, shape, dev) or _off(y, b16, shape, dev) or _off(codes, u8, shape, dev)
            or _off(exps, i8, (rows, pitch), dev)):
        _refuse(call, dev, x=(x, b16, shape), weight=(weight, b16, (K,)), residual=(residual, b16, shape),
                sum_out=(sum_out, b16, shape), y=(y, b16, shape), codes=(codes, u8, shape),
                exps=(exps, i8, (rows, pitch)))
    if residual is not None and sum_out is None:
        sum_out = _new(x, stream, shape, b16)
    if normed and y is None:
        y = _new(x, stream, shape, b16)
    if quantized and codes is None:
        codes = _new(x, stream, shape, u8)
    if quantized and exps is None:
        exps = _new(x, stream, (rows, pitch), i8)
    _run(call, dev, x.data_ptr(), _ptr(residual), weight.data_ptr(), rows, K, eps, _ptr(sum_out), _ptr(y),
         _ptr(codes), _ptr(exps), pitch, st)
    return sum_out, y, codes, exps


def moe_router_scores_workspace_size(T: int, H: int, E: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_router_scores_workspace_size",
           lib().moe_router_scores_workspace_size(T, H, E, ctypes.byref(n)))
    return n.value


def moe_router_scores(x, w, scores=None, ws=None, stream=None):
    """Router scores fp32 [T, E] of bf16 bits x [T, H] with w [E, H] (bf16 bits, torch.int16, or
    torch.float32).  `ws` (uint8 device tensor) is the call's workspace; None allocates one."""
    call = "moe_router_scores"
    if x.dim() != 2 or w.dim() != 2 or w.dtype not in (torch.int16, torch.float32):
        raise ValueError(f"{call}: x [T, H] and w [E, H] (torch.int16 or torch.float32) are wanted")
    dev, st = _where(call, x, stream)
    (T, H), E, f32 = x.shape, w.shape[0], torch.float32
    if (_off(x, torch.int16, (T, H), dev) or _off(w, w.dtype, (E, H), dev)
            or _off(scores, f32, (T, E), dev) or (ws is not None and _off(ws, torch.uint8, (ws.numel(),), dev))):
        _refuse(call, dev, x=(x, torch.int16, (T, H)), w=(w, w.dtype, (E, H)), scores=(scores, f32, (T, E)),
                ws=(ws, torch.uint8, None if ws is None else (ws.numel(),)))
    if scores is None:
        scores = _new(x, stream, (T, E), f32)
    if ws is None and T > 16:
        need = moe_router_scores_workspace_size(T, H, E)
        ws = _new(x, stream, (need,), torch.uint8) if need else None
    _run(call, dev, x.data_ptr(), T, H, w.data_ptr(), MOE_ROUTER_W_F32 if w.dtype is f32 else MOE_ROUTER_W_BF16,
         E, scores.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel(), st)
    return scores


def moe_linear_a8(codes, exps, w, s_w, y=None, stream=None):
    """y = x W^T as bf16 bits [M, N]: x quantised by moe_quantize_act or moe_rmsnorm_quantize_act (codes
    uint8 [M, K], exps int8 [M, pitch]), w uint8 [N, K] E4M3FN codes, s_w fp32 [ceil(N/128), K/128]."""
    call = "moe_linear_a8"
    if codes.dim() != 2 or w.dim() != 2 or exps.dim() != 2:
        raise ValueError(f"{call}: codes [M, K], exps [M, pitch] and w [N, K] are wanted")
    dev, st = _where(call, codes, stream)
    (M, K), N, pitch, u8, i8 = codes.shape, w.shape[0], exps.shape[1], torch.uint8, torch.int8
    blocks = (-(-N // 128), K // 128)
    if (_off(codes, u8, (M, K), dev) or _off(exps, i8, (M, pitch), dev) or _off(w, u8, (N, K), dev)
            or _off(s_w, torch.float32, blocks, dev) or _off(y, torch.int16, (M, N), dev)):
        _refuse(call, dev, codes=(codes, u8, (M, K)), exps=(exps, i8, (M, pitch)), w=(w, u8, (N, K)),
                s_w=(s_w, torch.float32, blocks), y=(y, torch.int16, (M, N)))
    if y is None:
        y = _new(codes, stream, (M, N), torch.int16)
    _run(call, dev, codes.data_ptr(), exps.data_ptr(), pitch, M, N, K, w.data_ptr(), s_w.data_ptr(),
         y.data_ptr(), st)
    return y


FEW_MAX_TOKENS = 8  # MOE_FEW_MAX_TOKENS
FEW_MAX_X = 57408   # moe_layer_few's limit on T * (H + 8)


def moe_layer_few_workspace_size(T: int, k: int, w: MoeExpertWeights) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_layer_few_workspace_size",
           lib().moe_layer_few_workspace_size(T, k, ctypes.byref(w), ctypes.byref(n)))
    return n.value


def moe_layer_few(scores, x, k: int, w: MoeExpertWeights, shared=None, score_fn="sigmoid",
                  renorm: int = 1, topk_ids=None, topk_w=None, out=None, work=None, stream=None):
    """The whole layer for up to FEW_MAX_TOKENS tokens in two launches; returns out (bf16 bits
    [T, H]), topk_ids and topk_w.  `shared` is the shared expert's MoeExpertWeights or None; `work`
    (uint8 device tensor) is the call's workspace, None allocates one."""
    call = "moe_layer_few"
    if x.dim() != 2 or scores.dim() != 2:
        raise ValueError(f"{call}: scores [T, E] and x [T, H] are wanted")
    dev, st = _where(call, x, stream)
    (T, H), E, i32, f32, b16 = x.shape, w.n_groups, torch.int32, torch.float32, torch.int16
    if H != w.H:
        raise ValueError(f"{call}: x has rows of {H}, the weights take {w.H}")
    if (_off(scores, f32, (T, E), dev) or _off(x, b16, (T, H), dev) or _off(topk_ids, i32, (T, k), dev)
            or _off(topk_w, f32, (T, k), dev) or _off(out, b16, (T, H), dev)
            or (work is not None and _off(work, torch.uint8, (work.numel(),), dev))):
        _refuse(call, dev, scores=(scores, f32, (T, E)), x=(x, b16, (T, H)), topk_ids=(topk_ids, i32, (T, k)),
                topk_w=(topk_w, f32, (T, k)), out=(out, b16, (T, H)),
                work=(work, torch.uint8, None if work is None else (work.numel(),)))
    fn = SCORE_FN[score_fn] if isinstance(score_fn, str) else int(score_fn)
    if topk_ids is None:
        topk_ids = _new(x, stream, (T, k), i32)
    if topk_w is None:
        topk_w = _new(x, stream, (T, k), f32)
    if out is None:
        out = _new(x, stream, (T, H), b16)
    if work is None:
        work = _new(x, stream, (moe_layer_few_workspace_size(T, k, w),), torch.uint8)
    _run(call, dev, scores.data_ptr(), x.data_ptr(), T, k, fn, int(renorm), ctypes.byref(w),
         None if shared is None else ctypes.byref(shared), topk_ids.data_ptr(), topk_w.data_ptr(),
         out.data_ptr(), work.data_ptr(), work.numel(), st)
    return out, topk_ids, topk_w


def _permute_ws(T, k, E, device):
    """moe_permute's workspace for T tokens (a 16-byte stand-in when none is needed)."""
    return torch.empty(max(16, moe_permute_workspace_size(T, k, E)), dtype=torch.uint8,
                       device=device)


class MoeLayer:
    """Buffers and the call sequence of one MoE layer forward: route -> permute (one launch,
    moe_route_permute, for T*k <= 2048) -> routed gate/up -> routed down -> combine on the
    caller's stream.  The shared expert (which only needs x) runs inside the routed launches at
    decode sizes (fuse_shared, below), and otherwise on a second stream that runs alongside the
    routed experts and joins before combine.

    `experts` and `shared` are objects accepted by expert_weights(); `x` is bf16 bits [T, H]
    (torch.int16) and `scores` fp32 [T, E], all on the GPU.

    fuse_shared: at decode sizes (T*k <= 32*E, bf16 activations) the shared expert can run inside
    the routed launches as an extra group (moe_expert_gate_up_shared / moe_expert_down_shared):
    one grid per phase, no second stream, no cross-stream waits; the extra group's tiles take the
    first workgroups, spread over the XCDs.  "auto" does so wherever it applies: the tiny layer
    0.035 against 0.092 ms a step, the DeepSeek-V3 decode layer 0.638 against 0.648 ms (FP8
    weights) and 0.363 against 0.372 ms (MXFP4) with the side stream.  True / False force it.
    `h`, `y`, `sh_h` and `sh_y` are then views of the shared buffers.

    overlap_shared=False runs the shared expert on the caller's stream after the routed experts
    instead of on the side stream (measured equal or slower at every layer size: the side stream
    fills CUs left idle by the routing kernels and by the routed GEMMs' last tiles).

    act="fp8" selects the FP8 activation mode (moe_expert_ffn_a8) for the routed and the shared
    experts; `h` then views the routed h inside the workspace, before its quantisation.

    few=True runs the layer as moe_layer_few: two launches, for up to FEW_MAX_TOKENS tokens with
    bf16 activations; there are no counts, offsets, permutation, h or y then, and the result is closer to
    the formula than the separate calls' (which round h and y), so not the same bits.

    capture(scores, x) records the forward into a HIP graph and replay() reruns it.
    """

    def __init__(self, T, H, I, E, k, experts, shared, score_fn="sigmoid", renorm=1, device="cuda",
                 overlap_shared=True, act="bf16", fuse_shared="auto", few=False):
        if act not in ("bf16", "fp8"):
            raise ValueError(f"act must be 'bf16' or 'fp8', not {act!r}")
        if few and act != "bf16":
            raise ValueError("few=True takes bf16 activations")
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.act = act
        self.score_fn, self.renorm = score_fn, renorm
        self.w = expert_weights(experts)
        self.ws_ = expert_weights(shared) if shared is not None else None
        self._keep = (experts, shared)
        d, i32 = device, torch.int32
        self.topk_ids = torch.empty((T, k), dtype=i32, device=d)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=d)
        self.few = bool(few)
        if self.few:
            self.ws = torch.empty(max(16, moe_layer_few_workspace_size(T, k, self.w)),
                                  dtype=torch.uint8, device=d)
            self.out = torch.empty((max(1, T), H), dtype=torch.int16, device=d)
            self.side, self.fused = None, False
            return
        self.counts = torch.empty(E, dtype=i32, device=d)
        self.offsets = torch.empty(E + 1, dtype=i32, device=d)
        self.perm = torch.empty(max(1, T * k), dtype=i32, device=d)
        self.inv = torch.empty(max(1, T * k), dtype=i32, device=d)
        self.perm_ws = _permute_ws(T, k, E, d)
        if act == "fp8":
            self.ws = torch.empty(max(1, moe_expert_ffn_a8_workspace_size(T, k, self.w)),
                                  dtype=torch.uint8, device=d)
            # h (before its quantisation) opens the workspace
            self.h = self.ws[:max(1, T * k) * I * 2].view(torch.int16).view(-1, I)
            self.sh_ws = self.sh_h = None
            if shared is not None:
                self.sh_ws = torch.empty(max(1, moe_expert_ffn_a8_workspace_size(T, 1, self.ws_)),
                                         dtype=torch.uint8, device=d)
                self.sh_h = self.sh_ws[:max(1, T) * I * 2].view(torch.int16).view(-1, I)
        # the shared expert as an extra group of the routed decode launches
        if fuse_shared == "auto":
            fuse_shared = True
        self.fused = (bool(fuse_shared) and act == "bf16" and shared is not None and T > 0
                      and T * k <= 32 * E and self.ws_.dtype == self.w.dtype
                      and self.ws_.H == self.w.H and self.ws_.I == self.w.I)
        if self.fused:
            self.h_all = torch.empty((T * k + T, I), dtype=torch.int16, device=d)
            self.y_all = torch.empty((T * k + T, H), dtype=torch.int16, device=d)
            self.h, self.sh_h = self.h_all[:T * k], self.h_all[T * k:]
            self.y, self.sh_y = self.y_all[:T * k], self.y_all[T * k:]
        else:
            if act != "fp8":
                self.h = torch.empty((max(1, T * k), I), dtype=torch.int16, device=d)
                self.sh_h = torch.empty((max(1, T), I), dtype=torch.int16, device=d)
            self.y = torch.empty((max(1, T * k), H), dtype=torch.int16, device=d)
            self.sh_y = torch.empty((max(1, T), H), dtype=torch.int16, device=d)
        self.out = torch.empty((max(1, T), H), dtype=torch.int16, device=d)
        self.side = (torch.cuda.Stream(device=d)
                     if (overlap_shared and shared is not None and not self.fused) else None)

    def capture(self, scores, x):
        """Record one forward on the tensors `scores` and `x` into a HIP graph; replay() reruns it
        on whatever they hold then.  None of the layer's calls allocates or clears memory, so the
        whole sequence (both streams) can be captured."""
        warm = torch.cuda.Stream()
        warm.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(warm):
            self.forward(scores, x)
        torch.cuda.current_stream().wait_stream(warm)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.forward(scores, x)
        return self.graph

    def replay(self):
        """Enqueue the captured forward on torch's current stream; returns `out`."""
        self.graph.replay()
        return self.out

    def _route_permute(self, scores, stream):
        """Routing and grouping; one launch for decode-sized batches."""
        k = self.k
        if self.T * k <= FUSED_ROUTE_PERMUTE_MAX:
            moe_route_permute(scores, k, self.score_fn, self.renorm, self.topk_ids, self.topk_w,
                              self.counts, self.offsets, self.perm, self.inv, stream)
        else:
            moe_route(scores, k, self.score_fn, self.renorm, self.topk_ids, self.topk_w, stream)
            moe_permute(self.topk_ids, self.E, self.counts, self.offsets, self.perm, self.inv,
                        self.perm_ws, stream)

    def _shared(self, x, st):
        if self.act == "fp8":
            moe_expert_ffn_a8(x, 1, None, None, self.ws_, self.sh_y, self.sh_ws, st)
        else:
            moe_expert_gate_up(x, 1, None, None, self.ws_, self.sh_h, st)
            moe_expert_down(self.sh_h, self.T, 1, None, self.ws_, self.sh_y, st)

    def forward(self, scores, x, stream=None, gate_up_events=None):
        """Enqueue the layer; returns `out` (bf16 bits [T, H]).  gate_up_events=(start, stop)
        records torch events around the routed gate/up kernel (for timing; bf16 mode only)."""
        T, k = self.T, self.k
        if self.few:
            if gate_up_events is not None:
                raise ValueError("few=True has no routed gate/up launch of its own")
            moe_layer_few(scores, x, k, self.w, self.ws_, self.score_fn, self.renorm, self.topk_ids,
                          self.topk_w, self.out[:T], self.ws, stream)
            return self.out
        main = torch.cuda.current_stream() if stream is None else stream
        shared_y = None
        if self.ws_ is not None and self.side is not None:
            # shared expert on the side stream, ordered after everything already on `main`
            self.side.wait_stream(main)
            self._shared(x, self.side)
            shared_y = self.sh_y
        self._route_permute(scores, stream)
        if self.fused:
            if gate_up_events is not None:  # (here the routed and the shared gate/up)
                gate_up_events[0].record(stream)
            moe_expert_gate_up_shared(x, k, self.perm, self.offsets, self.w, self.ws_, self.h_all,
                                      stream)
            if gate_up_events is not None:
                gate_up_events[1].record(stream)
            moe_expert_down_shared(self.h_all, T, k, self.offsets, self.w, self.ws_, self.y_all,
                                   stream)
            moe_combine(self.y, self.inv, self.topk_w, self.sh_y, T, k, self.H, self.out, stream)
            return self.out
        if self.act == "fp8":
            moe_expert_ffn_a8(x, k, self.perm, self.offsets, self.w, self.y, self.ws, stream)
        else:
            if gate_up_events is not None:
                gate_up_events[0].record(stream)
            moe_expert_gate_up(x, k, self.perm, self.offsets, self.w, self.h, stream)
            if gate_up_events is not None:
                gate_up_events[1].record(stream)
            moe_expert_down(self.h, T, k, self.offsets, self.w, self.y, stream)
        if self.ws_ is not None and self.side is None:
            self._shared(x, stream)
            shared_y = self.sh_y
        elif self.side is not None:
            main.wait_stream(self.side)
        moe_combine(self.y, self.inv, self.topk_w, shared_y, T, k, self.H, self.out, stream)
        return self.out


class MoeBlock:
    """Buffers and the call sequence of the second half of a transformer block whose feed-forward part is
    a MoE layer:
        s = hidden + residual;  n = RMS norm of s;  scores = n router_w^T;  out = the layer of n
    moe_rmsnorm_quantize_act -> moe_router_scores -> MoeLayer, on the caller's stream (the layer's
    shared expert as MoeLayer places it).  The next block's norm adds `out` to s.

    `norm_w` is bf16 bits [H], `router_w` [E, H] bf16 bits or fp32; the other arguments are MoeLayer's.

    act="fp8" with many rows per expert (T*k > 32*E, FP8 or MXFP4 weights, H a multiple of 256 and H and
    I at most 8192): the gate/up GEMMs of the routed and the shared experts take the norm's own codes
    (moe_expert_gate_up_a8), so that x is not read and quantised once more by each of them, and the codes
    are those of the norm before its rounding to bf16.  Otherwise the layer quantises `normed` itself.

    few="auto" (act="bf16") runs the layer as moe_layer_few wherever it takes the sizes; True / False
    force it.

    forward(hidden, residual) returns (out, s), capture(hidden, residual) records it into a HIP graph.
    `residual` may be None (then s is hidden itself).
    """

    def __init__(self, T, H, I, E, k, norm_w, router_w, experts, shared, eps=1e-6,
                 score_fn="sigmoid", renorm=1, device="cuda", act="bf16", few="auto"):
        if few == "auto":
            few = act == "bf16" and T <= FEW_MAX_TOKENS and T * (H + 8) <= FEW_MAX_X and k <= 32
        self.layer = MoeLayer(T, H, I, E, k, experts, shared, score_fn, renorm, device, act=act, few=few)
        self.T, self.H, self.E, self.k, self.eps = T, H, E, k, eps
        self.norm_w, self.router_w = norm_w, router_w
        d, b16 = device, torch.int16
        self.sum = torch.empty((T, H), dtype=b16, device=d)
        self.normed = torch.empty((T, H), dtype=b16, device=d)
        self.scores = torch.empty((T, E), dtype=torch.float32, device=d)
        self.router_ws = torch.empty(max(16, moe_router_scores_workspace_size(T, H, E)),
                                     dtype=torch.uint8, device=d)
        L = self.layer
        self.codes = None
        if (act == "fp8" and T * k > 32 * E and T > 32 and L.w.dtype != MOE_W_BF16 and H % 256 == 0
                and H <= 8192 and I <= 8192 and (L.ws_ is None or L.ws_.dtype != MOE_W_BF16)):
            def quantised(rows, K):
                return (torch.empty((rows, K), dtype=torch.uint8, device=d),
                        torch.empty((rows, exp_pitch(K)), dtype=torch.int8, device=d))
            self.codes, self.exps = quantised(T, H)
            self.h_q = quantised(T * k, I)
            self.sh_q = quantised(T, I) if shared is not None else None

    def _layer_a8(self, stream):
        """The layer in the FP8 mode on the norm's codes, the shared expert on the layer's side stream."""
        L, T, k = self.layer, self.T, self.k
        main = torch.cuda.current_stream() if stream is None else stream
        if L.side is not None:
            L.side.wait_stream(main)
            self._experts_a8(1, None, None, L.ws_, L.sh_h, self.sh_q, L.sh_y, L.side)
        L._route_permute(self.scores, stream)
        self._experts_a8(k, L.perm, L.offsets, L.w, L.h, self.h_q, L.y, stream)
        if L.side is not None:
            main.wait_stream(L.side)
        moe_combine(L.y, L.inv, L.topk_w, L.sh_y if L.side is not None else None, T, k, self.H, L.out,
                    stream)
        return L.out

    def _experts_a8(self, k, perm, offsets, w, h, h_q, y, stream):
        moe_expert_gate_up_a8(self.codes, self.exps, k, perm, offsets, w, h, stream)
        moe_quantize_act(h, *h_q, h_q[1].shape[1], stream)
        moe_expert_down_a8(*h_q, self.T, k, offsets, w, y, stream)

    def forward(self, hidden, residual=None, stream=None):
        """Enqueue the block; returns (out, s), bf16 bits [T, H] (buffers of the block, `hidden` as s
        without a residual)."""
        a8 = self.codes is not None
        moe_rmsnorm_quantize_act(hidden, self.norm_w, residual, self.eps, quantized=a8,
                                 sum_out=None if residual is None else self.sum, y=self.normed,
                                 codes=self.codes, exps=self.exps if a8 else None, stream=stream)
        moe_router_scores(self.normed, self.router_w, self.scores, self.router_ws, stream)
        out = self._layer_a8(stream) if a8 else self.layer.forward(self.scores, self.normed, stream)
        return out[:self.T], hidden if residual is None else self.sum

    def capture(self, hidden, residual=None):
        """Record one forward on the tensors `hidden` and `residual` into a HIP graph; replay() reruns it
        on whatever they hold then."""
        warm = torch.cuda.Stream()
        warm.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(warm):
            self.forward(hidden, residual)
        torch.cuda.current_stream().wait_stream(warm)
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self._result = self.forward(hidden, residual)
        return self.graph

    def replay(self):
        """Enqueue the captured forward on torch's current stream; returns (out, s)."""
        self.graph.replay()
        return self._result


class MoeRankShare:
    """One rank's share of the layer under expert parallelism over G ranks, as in the SmallEP
    scheme of the OSDI'26 hybrid-inference article (SmallEP section): after the tokens are
    all-gathered, every rank routes and groups all T tokens (redundantly), runs its local routed
    experts [e_begin, e_end) on the assignments that select them, and reduces their weighted
    outputs to a partial [T, H] (moe_combine_partial); the partials are then exchanged and
    summed.  The shared expert runs on the rank's own token rows [t_begin, t_end).

    `experts` holds all E experts' weights (only the local slice is ever read: expert_slice);
    forward() returns (partial [T, H], shared output [t_end - t_begin, H]), bf16 bits.  The
    collectives are not part of this single-GPU build.
    """

    def __init__(self, T, H, I, E, k, experts, shared, e_begin, e_end, t_begin, t_end,
                 score_fn="sigmoid", renorm=1, device="cuda"):
        if not (0 <= e_begin <= e_end <= E and 0 <= t_begin <= t_end <= T):
            raise ValueError("expert or token range out of bounds")
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.e0, self.e1, self.t0, self.t1 = e_begin, e_end, t_begin, t_end
        self.score_fn, self.renorm = score_fn, renorm
        local = expert_slice(experts, e_begin, e_end)
        self.w = expert_weights(local) if e_end > e_begin else None
        self.ws_ = expert_weights(shared) if shared is not None else None
        self._keep = (experts, shared, local)
        d, i32 = device, torch.int32
        self.topk_ids = torch.empty((T, k), dtype=i32, device=d)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=d)
        self.counts = torch.empty(E, dtype=i32, device=d)
        self.offsets = torch.empty(E + 1, dtype=i32, device=d)
        self.perm = torch.empty(max(1, T * k), dtype=i32, device=d)
        self.inv = torch.empty(max(1, T * k), dtype=i32, device=d)
        self.perm_ws = _permute_ws(T, k, E, d)
        self.h = torch.empty((max(1, T * k), I), dtype=torch.int16, device=d)
        self.y = torch.empty((max(1, T * k), H), dtype=torch.int16, device=d)
        self.out = torch.empty((max(1, T), H), dtype=torch.int16, device=d)
        nt = max(1, t_end - t_begin)
        self.sh_h = torch.empty((nt, I), dtype=torch.int16, device=d)
        self.sh_y = torch.empty((nt, H), dtype=torch.int16, device=d)

    def forward(self, scores, x, stream=None, gate_up_events=None):
        T, k = self.T, self.k
        if T * k <= FUSED_ROUTE_PERMUTE_MAX:
            moe_route_permute(scores, k, self.score_fn, self.renorm, self.topk_ids, self.topk_w,
                              self.counts, self.offsets, self.perm, self.inv, stream)
        else:
            moe_route(scores, k, self.score_fn, self.renorm, self.topk_ids, self.topk_w, stream)
            moe_permute(self.topk_ids, self.E, self.counts, self.offsets, self.perm, self.inv,
                        self.perm_ws, stream)
        if self.w is not None:
            offs = self.offsets[self.e0:]  # the local experts' slice of the grouping
            if gate_up_events is not None:
                gate_up_events[0].record(stream)
            moe_expert_gate_up(x, k, self.perm, offs, self.w, self.h, stream)
            if gate_up_events is not None:
                gate_up_events[1].record(stream)
            moe_expert_down(self.h, T, k, offs, self.w, self.y, stream)
        moe_combine_partial(self.y, self.inv, self.topk_ids, self.topk_w, self.e0, self.e1, None,
                            T, k, self.H, self.out, stream)
        if self.ws_ is not None and self.t1 > self.t0:
            xs = x[self.t0:self.t1]
            moe_expert_gate_up(xs, 1, None, None, self.ws_, self.sh_h, stream)
            moe_expert_down(self.sh_h, self.t1 - self.t0, 1, None, self.ws_, self.sh_y, stream)
        return self.out, self.sh_y

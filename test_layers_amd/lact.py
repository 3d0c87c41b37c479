"""Thin ctypes binding of liblact (include/lact.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Torch tensors supply device memory (data_ptr) and the current HIP
stream; nothing here computes any part of the layer.  If liblact.so is
missing the import fails loudly -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import operator
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblact.so")

# values mirror include/lact.h
OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED = -2
ERR_WORKSPACE_TOO_SMALL = -3
ERR_NO_DEVICE = -4
ERR_HIP = -5

DTYPE_F32 = 0
DTYPE_BF16 = 1
OPT_GD = 0
OPT_MOMENTUM = 1
OPT_MUON = 2
OPT_MUON_MOMENTUM = 3
APPLY_THEN_UPDATE = 0
UPDATE_THEN_APPLY = 1
CHUNK_UPDATE = 1
CHUNK_APPLY = 2
NO_RENORM = 1
QK_PREP = 2

ROTARY_INTERLEAVED = 1
ROTARY_INVERSE = 2
ROTARY_SCALING = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}
CLEAR_REST = 1
NORM_GROUP = 128   # LACT_NORM_GROUP: columns that share a scale of the 8-bit output

(K_UPD, K_APP, K_OUT, K_DW, K_OPT, K_NS, K_SNAP, K_PREP, K_BWD_GEMM, K_BWD_ELEM, K_NSRED, K_ATTN, K_ATTN_BWD,
 K_ROTARY, K_NORM, K_PAGES) = range(16)
K_NAMES = {K_UPD: "update_fwd", K_APP: "apply_fwd", K_OUT: "apply_out", K_DW: "dw", K_OPT: "opt",
           K_NS: "newton_schulz", K_SNAP: "snapshot", K_PREP: "qk_prep", K_BWD_GEMM: "bwd_gemm",
           K_BWD_ELEM: "bwd_elem", K_NSRED: "ns_reduce", K_ATTN: "attention", K_ATTN_BWD: "attention_bwd",
           K_ROTARY: "rotary", K_NORM: "norm", K_PAGES: "pages"}

EXPORTS = ["lact_workspace_size", "lact_chunk_update", "lact_apply", "lact_layer_forward",
           "lact_layer_forward_scaled", "lact_layer_forward_noalloc", "lact_backward_workspace_size",
           "lact_layer_backward", "lact_window_attention_workspace_size", "lact_window_attention_forward",
           "lact_window_attention_backward_workspace_size", "lact_window_attention_backward", "lact_rotary",
           "lact_rotary_frequencies", "lact_add_rmsnorm_forward", "lact_add_rmsnorm_backward_workspace_size",
           "lact_add_rmsnorm_backward", "lact_packed_attention_forward",
           "lact_packed_attention_backward_workspace_size", "lact_packed_attention_backward",
           "lact_paged_attention_workspace_size", "lact_paged_attention", "lact_page_slots_workspace_size",
           "lact_page_slots", "lact_page_write", "lact_status_str", "lact_last_error", "lact_timing_enable", "lact_timing_read"]

NOALLOC_SCRATCH_BYTES = 128 << 20   # LACT_NOALLOC_SCRATCH_BYTES


class LactError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"liblact status {status}: {detail}")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [("n_inst", ctypes.c_int32), ("d", ctypes.c_int32), ("dh", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("opt", ctypes.c_int32), ("ns_iters", ctypes.c_int32),
                ("rec_planes", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class Strides(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("token", ctypes.c_int64)]


class Attention(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_len", ctypes.c_int64), ("k_len", ctypes.c_int64), ("window", ctypes.c_int64),
                ("sinks", ctypes.c_int64)]


class RotaryProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("pairs", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("mscale", ctypes.c_float), ("tokens", ctypes.c_int64),
                ("start", ctypes.c_int64)]


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class Packed(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("tokens", ctypes.c_int64), ("longest", ctypes.c_int64), ("window", ctypes.c_int64),
                ("sinks", ctypes.c_int64), ("flags", ctypes.c_uint32)]


class Paged(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("tokens", ctypes.c_int64), ("longest", ctypes.c_int64), ("k_len", ctypes.c_int64),
                ("window", ctypes.c_int64), ("sinks", ctypes.c_int64), ("pages", ctypes.c_int32),
                ("page", ctypes.c_int32), ("width", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class Slots(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("page", ctypes.c_int32), ("width", ctypes.c_int32),
                ("entries", ctypes.c_int32), ("tokens", ctypes.c_int64)]


class Write(ctypes.Structure):
    _fields_ = [("kv_heads", ctypes.c_int32), ("d", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("pages", ctypes.c_int32), ("page", ctypes.c_int32), ("tokens", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m test_layers_amd.build` "
                          "(the LaCT layer has no non-HIP implementation)")
    # torch ships its own HIP runtime, reached through the unversioned name
    # libamdhip64.so.  If liblact were loaded first, its dependency
    # libamdhip64.so.7 would resolve to the system runtime and the process
    # would hold two HIP (and HSA) runtimes; the second one to open the GPU
    # sees no device.  Loading torch first makes liblact bind to the runtime
    # that owns the tensors it is given.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    P = ctypes.POINTER(Problem)
    L.lact_workspace_size.restype = sz
    L.lact_workspace_size.argtypes = [P, i64, i64, i32, vp, vp, i32]
    L.lact_chunk_update.restype = i32
    L.lact_chunk_update.argtypes = [P, vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lact_apply.restype = i32
    L.lact_apply.argtypes = [P, vp, i64, i64, vp, vp, vp, vp, vp, sz, vp]
    L.lact_layer_forward.restype = i32
    L.lact_layer_forward.argtypes = [P, vp, vp, vp, vp, vp, i64, i64, i32, vp, vp, i32,
                                     vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lact_layer_forward_scaled.restype = i32
    L.lact_layer_forward_scaled.argtypes = [P, vp, vp, vp, vp, vp, vp, i64, i64, i32, vp, vp, i32,
                                            vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.lact_layer_forward_noalloc.restype = i32
    L.lact_layer_forward_noalloc.argtypes = [P, vp, vp, vp, vp, vp, i64, i64, i32, vp, vp, i32,
                                             vp, vp, vp, vp, vp, vp, vp, vp]
    L.lact_backward_workspace_size.restype = sz
    L.lact_backward_workspace_size.argtypes = [P, i64, i64, i32, vp, vp, i32]
    L.lact_layer_backward.restype = i32
    L.lact_layer_backward.argtypes = ([P, vp, vp, vp, vp, vp, vp, i64, i64, i32, vp, vp, i32]
                                      + [vp] * 6 + [vp] + [vp] * 6 + [vp] * 6 + [vp] * 6 + [vp, sz, vp])
    A, R, N, f64 = ctypes.POINTER(Attention), ctypes.POINTER(RotaryProblem), ctypes.POINTER(NormProblem), ctypes.c_double
    L.lact_window_attention_workspace_size.restype = sz
    L.lact_window_attention_workspace_size.argtypes = [A]
    L.lact_window_attention_forward.restype = i32
    L.lact_window_attention_forward.argtypes = [A] + [vp] * 12 + [sz, vp]
    L.lact_window_attention_backward_workspace_size.restype = sz
    L.lact_window_attention_backward_workspace_size.argtypes = [A]
    L.lact_window_attention_backward.restype = i32
    L.lact_window_attention_backward.argtypes = [A] + [vp] * 20 + [sz, vp]
    L.lact_rotary.restype = i32
    L.lact_rotary.argtypes = [R] + [vp] * 11
    L.lact_rotary_frequencies.restype = i32
    L.lact_rotary_frequencies.argtypes = [i32, f64, i32, f64, i64, f64, f64, vp, ctypes.POINTER(ctypes.c_float)]
    L.lact_add_rmsnorm_forward.restype = i32
    L.lact_add_rmsnorm_forward.argtypes = [N, vp, i64, vp, i64, vp, vp, i64, vp, i64, vp, i64, vp, vp]
    L.lact_add_rmsnorm_backward_workspace_size.restype = sz
    L.lact_add_rmsnorm_backward_workspace_size.argtypes = [N]
    L.lact_add_rmsnorm_backward.restype = i32
    L.lact_add_rmsnorm_backward.argtypes = [N, vp, i64, vp, vp, i64, vp, i64, vp, i64, vp, vp, sz, vp]
    K, G, S, W = (ctypes.POINTER(x) for x in (Packed, Paged, Slots, Write))
    L.lact_packed_attention_forward.restype = i32
    L.lact_packed_attention_forward.argtypes = [K] + [vp] * 11
    L.lact_packed_attention_backward_workspace_size.restype = sz
    L.lact_packed_attention_backward_workspace_size.argtypes = [K]
    L.lact_packed_attention_backward.restype = i32
    L.lact_packed_attention_backward.argtypes = [K] + [vp] * 19 + [sz, vp]
    L.lact_paged_attention_workspace_size.restype = sz
    L.lact_paged_attention_workspace_size.argtypes = [G]
    L.lact_paged_attention.restype = i32
    L.lact_paged_attention.argtypes = [G] + [vp] * 13 + [sz, vp]
    L.lact_page_slots_workspace_size.restype = sz
    L.lact_page_slots_workspace_size.argtypes = [S]
    L.lact_page_slots.restype = i32
    L.lact_page_slots.argtypes = [S] + [vp] * 11 + [sz, vp]
    L.lact_page_write.restype = i32
    L.lact_page_write.argtypes = [W] + [vp] * 10
    L.lact_status_str.restype = ctypes.c_char_p
    L.lact_status_str.argtypes = [i32]
    L.lact_last_error.restype = ctypes.c_char_p
    L.lact_last_error.argtypes = []
    L.lact_timing_enable.restype = i32
    L.lact_timing_enable.argtypes = [i32, i32]
    L.lact_timing_read.restype = i32
    L.lact_timing_read.argtypes = [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
    _lib = L
    return L


def last_error() -> str:
    return lib().lact_last_error().decode()


def check(status: int) -> None:
    if status != OK:
        raise LactError(status, f"{lib().lact_status_str(status).decode()}: {last_error()}")


def problem(n_inst: int, d: int, io_dtype: int, opt: int, rec_planes: int = 0, ns_iters: int = 5,
            renorm: bool = True, dh: Optional[int] = None, qk_prep: bool = False) -> Problem:
    return Problem(n_inst, d, d if dh is None else dh, io_dtype, opt, ns_iters, rec_planes,
                   (0 if renorm else NO_RENORM) | (QK_PREP if qk_prep else 0))


# ----------------------------------------------------------------- raw-pointer calls
_SCHED_CACHE = {}


def _sched(bounds, flags):
    # either may be None: the library reports a half-given schedule itself.
    # Both given: the library reads n_chunks + 1 bounds and n_chunks flags,
    # so their lengths must agree, and flags must fit the uint8 they become.
    # A layer call marshals its schedule twice (workspace size, then the
    # call), and callers repeat schedules: the converted arrays of recent
    # schedules are kept (they are read by the library only during a call).
    if bounds is None and flags is None:
        return None, None, 0, None
    key = (None if bounds is None else tuple(bounds), None if flags is None else tuple(flags))
    hit = _SCHED_CACHE.get(key)
    if hit is not None:
        return hit
    res = _sched_convert(bounds, flags)
    if len(_SCHED_CACHE) >= 64:
        _SCHED_CACHE.clear()
    _SCHED_CACHE[key] = res
    return res


def _sched_convert(bounds, flags):
    if bounds is not None and flags is not None and len(bounds) != len(flags) + 1:
        raise ValueError(f"schedule has {len(bounds)} bounds for {len(flags)} chunks (need chunks + 1)")
    if flags is not None and any(not 0 <= int(x) <= 255 for x in flags):
        raise ValueError("schedule flags must lie in 0..255")
    b = None if bounds is None else (ctypes.c_int64 * len(bounds))(*[int(x) for x in bounds])
    f = None if flags is None else (ctypes.c_uint8 * len(flags))(*[int(x) for x in flags])
    nc = len(flags) if flags is not None else len(bounds) - 1
    cast = lambda a: None if a is None else ctypes.cast(a, ctypes.c_void_p)
    return cast(b), cast(f), nc, (b, f)


def workspace_size(p: Problem, L: int, chunk: int = 0, order: int = 0,
                   bounds: Optional[Sequence[int]] = None, flags: Optional[Sequence[int]] = None) -> int:
    bp, fp, nc, _keep = _sched(bounds, flags)
    n = lib().lact_workspace_size(ctypes.byref(p), L, chunk, order, bp, fp, nc)
    if n == 0:
        raise LactError(ERR_INVALID_ARG, last_error())
    return n


def layer_forward_ptr(p: Problem, q, k, v, lr, beta, L, chunk, order, bounds, flags,
                      W1, W2, W3, M1, M2, M3, o, ws, ws_bytes, stream) -> int:
    bp, fp, nc, _keep = _sched(bounds, flags)
    return lib().lact_layer_forward(ctypes.byref(p), q, k, v, lr, beta, L, chunk, order, bp, fp, nc,
                                    W1, W2, W3, M1, M2, M3, o, ws, ws_bytes, stream)


def layer_forward_scaled_ptr(p: Problem, q, k, v, lr, beta, oz, L, chunk, order, bounds, flags,
                             W1, W2, W3, M1, M2, M3, o, ws, ws_bytes, stream) -> int:
    bp, fp, nc, _keep = _sched(bounds, flags)
    return lib().lact_layer_forward_scaled(ctypes.byref(p), q, k, v, lr, beta, oz, L, chunk, order,
                                           bp, fp, nc, W1, W2, W3, M1, M2, M3, o, ws, ws_bytes, stream)


def layer_forward_noalloc_ptr(p: Problem, q, k, v, lr, beta, L, chunk, order, bounds, flags,
                              W1, W2, W3, M1, M2, M3, o, stream) -> int:
    bp, fp, nc, _keep = _sched(bounds, flags)
    return lib().lact_layer_forward_noalloc(ctypes.byref(p), q, k, v, lr, beta, L, chunk, order, bp, fp, nc,
                                            W1, W2, W3, M1, M2, M3, o, stream)


def backward_workspace_size(p: Problem, L: int, chunk: int = 0, order: int = 0,
                            bounds: Optional[Sequence[int]] = None, flags: Optional[Sequence[int]] = None) -> int:
    bp, fp, nc, _keep = _sched(bounds, flags)
    n = lib().lact_backward_workspace_size(ctypes.byref(p), L, chunk, order, bp, fp, nc)
    if n == 0:
        raise LactError(ERR_INVALID_ARG, last_error())
    return n


def layer_backward_ptr(p: Problem, q, k, v, lr, beta, oz, L, chunk, order, bounds, flags, W1, W2, W3, M1, M2, M3,
                       dO, gW1, gW2, gW3, gM1, gM2, gM3, dq, dk, dv, dlr, dbeta, doz, dW1, dW2, dW3, dM1, dM2, dM3,
                       ws, ws_bytes, stream) -> int:
    bp, fp, nc, _keep = _sched(bounds, flags)
    return lib().lact_layer_backward(ctypes.byref(p), q, k, v, lr, beta, oz, L, chunk, order, bp, fp, nc,
                                     W1, W2, W3, M1, M2, M3, dO, gW1, gW2, gW3, gM1, gM2, gM3,
                                     dq, dk, dv, dlr, dbeta, doz, dW1, dW2, dW3, dM1, dM2, dM3, ws, ws_bytes,
                                     stream)


def chunk_update_ptr(p: Problem, k, v, lr, beta, Lc, seq_stride, W1, W2, W3, M1, M2, M3,
                     ws, ws_bytes, stream) -> int:
    return lib().lact_chunk_update(ctypes.byref(p), k, v, lr, beta, Lc, seq_stride, W1, W2, W3,
                                   M1, M2, M3, ws, ws_bytes, stream)


def apply_ptr(p: Problem, q, Lq, seq_stride, W1, W2, W3, o, ws, ws_bytes, stream) -> int:
    return lib().lact_apply(ctypes.byref(p), q, Lq, seq_stride, W1, W2, W3, o, ws, ws_bytes, stream)


def timing_enable(kclass: int, on: bool = True) -> None:
    check(lib().lact_timing_enable(kclass, 1 if on else 0))


def timing_read(kclass: int):
    ms = ctypes.c_double(0)
    n = ctypes.c_int64(0)
    check(lib().lact_timing_read(kclass, ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


# ----------------------------------------------------------------- torch-tensor calls
def _torch():
    import torch
    return torch


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    torch = _torch()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    return t.data_ptr()


def _check_shapes(**named):
    """Every given tensor must have exactly the expected shape: the library
    receives raw pointers and cannot detect a mis-sized buffer itself."""
    for name, (t, shape) in named.items():
        if t is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _w_shapes(n, D, Dh):
    return (n, Dh, D), (n, D, Dh), (n, Dh, D)


def _io_dtype(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise ValueError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _workspace(nbytes, workspace, device):
    torch = _torch()
    if workspace is not None:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or not workspace.is_cuda:
            raise ValueError("workspace must be a contiguous uint8 device tensor")
        if workspace.numel() < nbytes:
            raise ValueError(f"workspace smaller than the {nbytes} bytes needed")
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def layer_forward(q, k, v, lr, beta, W1, W2, W3, M1=None, M2=None, M3=None, o=None, *,
                  chunk: int = 0, order: int = APPLY_THEN_UPDATE, opt: int = OPT_GD,
                  bounds=None, flags=None, rec_planes: int = 0, ns_iters: int = 5,
                  renorm: bool = True, qk_prep: bool = False, oz=None, workspace=None,
                  stream=None):
    """q, k, v [n, L, d] (fp32 or bf16), lr [n, L, 3] fp32, beta [n, L] fp32
    (momentum) or None, W1, W3 [n, dh, d] and W2 [n, d, dh] fp32 (updated in
    place; dh is read from W1's shape), M1..M3
    (momentum state, updated in place).  qk_prep: q and k are raw (the library
    applies silu and the per-token L2 normalisation).  oz [n, L] fp32: the
    output rows are scaled by silu(oz) (lact_layer_forward_scaled).  Returns o
    [n, L, D] (allocated with torch.zeros if not given; rows of non-APPLY
    chunks keep their values)."""
    torch = _torch()
    if q.dim() != 3 or W1.dim() != 3:
        raise ValueError("q must be [n, L, d] and W1 [n, dh, d]")
    n, L, D = q.shape
    Dh = W1.shape[1]
    s1, s2, s3 = _w_shapes(n, D, Dh)
    _check_shapes(k=(k, (n, L, D)), v=(v, (n, L, D)), lr=(lr, (n, L, 3)), beta=(beta, (n, L)), W1=(W1, s1),
                  W2=(W2, s2), W3=(W3, s3), M1=(M1, s1), M2=(M2, s2), M3=(M3, s3), o=(o, (n, L, D)),
                  oz=(oz, (n, L)))
    io = _io_dtype(q)
    p = problem(n, D, io, opt, rec_planes, ns_iters, renorm, dh=Dh, qk_prep=qk_prep)
    if o is None:
        o = torch.zeros_like(q)
    need = workspace_size(p, L, chunk, order, bounds, flags)
    ws = _workspace(need, workspace, q.device)
    f32 = torch.float32
    head = (p, _ptr(q, q.dtype, "q"), _ptr(k, q.dtype, "k"), _ptr(v, q.dtype, "v"),
            _ptr(lr, f32, "lr"), _ptr(beta, f32, "beta"))
    tail = (L, chunk, order, bounds, flags,
            _ptr(W1, f32, "W1"), _ptr(W2, f32, "W2"), _ptr(W3, f32, "W3"),
            _ptr(M1, f32, "M1"), _ptr(M2, f32, "M2"), _ptr(M3, f32, "M3"),
            _ptr(o, q.dtype, "o"), ws.data_ptr(), ws.numel(), _stream(stream))
    if oz is None:
        st = layer_forward_ptr(*head, *tail)
    else:
        st = layer_forward_scaled_ptr(*head, _ptr(oz, f32, "oz"), *tail)
    check(st)
    return o


def chunk_update(k, v, lr, beta, W1, W2, W3, M1=None, M2=None, M3=None, *, Lc: Optional[int] = None,
                 opt: int = OPT_GD, rec_planes: int = 0, ns_iters: int = 5, renorm: bool = True,
                 qk_prep: bool = False, workspace=None, stream=None):
    torch = _torch()
    if k.dim() != 3 or W1.dim() != 3:
        raise ValueError("k must be [n, S, d] and W1 [n, dh, d]")
    n, S, D = k.shape
    s1, s2, s3 = _w_shapes(n, D, W1.shape[1])
    _check_shapes(v=(v, (n, S, D)), lr=(lr, (n, S, 3)), beta=(beta, (n, S)), W2=(W2, s2), W3=(W3, s3),
                  M1=(M1, s1), M2=(M2, s2), M3=(M3, s3))
    Lc = S if Lc is None else Lc
    p = problem(n, D, _io_dtype(k), opt, rec_planes, ns_iters, renorm, dh=W1.shape[1], qk_prep=qk_prep)
    ws = _workspace(workspace_size(p, Lc, max(Lc, 1)), workspace, k.device)
    f32 = torch.float32
    check(chunk_update_ptr(p, _ptr(k, k.dtype, "k"), _ptr(v, k.dtype, "v"), _ptr(lr, f32, "lr"),
                           _ptr(beta, f32, "beta"), Lc, S, _ptr(W1, f32, "W1"), _ptr(W2, f32, "W2"),
                           _ptr(W3, f32, "W3"), _ptr(M1, f32, "M1"), _ptr(M2, f32, "M2"),
                           _ptr(M3, f32, "M3"), ws.data_ptr(), ws.numel(), _stream(stream)))


def apply(q, W1, W2, W3, o=None, *, Lq: Optional[int] = None, qk_prep: bool = False,
          workspace=None, stream=None):
    torch = _torch()
    if q.dim() != 3 or W1.dim() != 3:
        raise ValueError("q must be [n, S, d] and W1 [n, dh, d]")
    n, S, D = q.shape
    s1, s2, s3 = _w_shapes(n, D, W1.shape[1])
    _check_shapes(W2=(W2, s2), W3=(W3, s3), o=(o, (n, S, D)))
    Lq = S if Lq is None else Lq
    p = problem(n, D, _io_dtype(q), OPT_GD, dh=W1.shape[1], qk_prep=qk_prep)
    if o is None:
        o = torch.zeros_like(q)
    ws = _workspace(workspace_size(p, Lq, max(Lq, 1)), workspace, q.device)
    f32 = torch.float32
    check(apply_ptr(p, _ptr(q, q.dtype, "q"), Lq, S, _ptr(W1, f32, "W1"), _ptr(W2, f32, "W2"),
                    _ptr(W3, f32, "W3"), _ptr(o, q.dtype, "o"), ws.data_ptr(), ws.numel(),
                    _stream(stream)))
    return o


def layer_backward(q, k, v, lr, beta, W1, W2, W3, M1=None, M2=None, M3=None, *, dO, gW=None, gM=None,
                   chunk: int = 0, order: int = APPLY_THEN_UPDATE, opt: int = OPT_GD, bounds=None, flags=None,
                   ns_iters: int = 5, renorm: bool = True, qk_prep: bool = False, oz=None, out=None,
                   workspace=None, stream=None):
    """Backward of layer_forward (lact_layer_backward).  Inputs as for
    layer_forward with W1..W3, M1..M3 the INITIAL state (read only); dO
    [n, L, d] in q's dtype (the cotangent of the scaled output when oz is
    given); gW, gM: None or 3-tuples of cotangents of the final state.
    Returns a dict of fp32 gradients dq, dk, dv (of the raw q, k with
    qk_prep), dlr, dbeta (momentum optimisers, else None), doz (with oz, else
    None), dW1..dW3, dM1..dM3 (momentum optimisers, else None); `out` (such a
    dict from an earlier call with the same shapes) is filled instead of
    allocating."""
    torch = _torch()
    if q.dim() != 3 or W1.dim() != 3:
        raise ValueError("q must be [n, L, d] and W1 [n, dh, d]")
    n, L, D = q.shape
    Dh = W1.shape[1]
    ws_ = _w_shapes(n, D, Dh)
    _check_shapes(k=(k, (n, L, D)), v=(v, (n, L, D)), lr=(lr, (n, L, 3)), beta=(beta, (n, L)), W2=(W2, ws_[1]),
                  W3=(W3, ws_[2]), M1=(M1, ws_[0]), M2=(M2, ws_[1]), M3=(M3, ws_[2]), dO=(dO, (n, L, D)),
                  oz=(oz, (n, L)))
    for name, gs in (("gW", gW), ("gM", gM)):
        for j, g in enumerate(gs or ()):
            _check_shapes(**{f"{name}{j + 1}": (g, ws_[j])})
    if out is not None:
        expect = {"dq": (n, L, D), "dk": (n, L, D), "dv": (n, L, D), "dlr": (n, L, 3), "dbeta": (n, L),
                  "doz": (n, L), "dW1": ws_[0], "dW2": ws_[1], "dW3": ws_[2], "dM1": ws_[0], "dM2": ws_[1],
                  "dM3": ws_[2]}
        _check_shapes(**{f"out[{key}]": (out.get(key), shape) for key, shape in expect.items()})
    io = _io_dtype(q)
    p = problem(n, D, io, opt, 3, ns_iters, renorm, dh=Dh, qk_prep=qk_prep)
    mom = opt in (OPT_MOMENTUM, OPT_MUON_MOMENTUM)
    f32 = torch.float32
    if out is None:
        e = lambda *shape: torch.empty(*shape, dtype=f32, device=q.device)
        out = {"dq": e(n, L, D), "dk": e(n, L, D), "dv": e(n, L, D), "dlr": e(n, L, 3),
               "dbeta": e(n, L) if mom else None, "doz": e(n, L) if oz is not None else None}
        for j, w in enumerate((W1, W2, W3)):
            out[f"dW{j + 1}"] = torch.empty_like(w)
            out[f"dM{j + 1}"] = torch.empty_like(w) if mom else None
    gW = (None, None, None) if gW is None else gW
    gM = (None, None, None) if gM is None else gM
    need = backward_workspace_size(p, L, chunk, order, bounds, flags)
    ws = _workspace(need, workspace, q.device)
    check(layer_backward_ptr(
        p, _ptr(q, q.dtype, "q"), _ptr(k, q.dtype, "k"), _ptr(v, q.dtype, "v"), _ptr(lr, f32, "lr"),
        _ptr(beta, f32, "beta"), _ptr(oz, f32, "oz"), L, chunk, order, bounds, flags,
        _ptr(W1, f32, "W1"), _ptr(W2, f32, "W2"), _ptr(W3, f32, "W3"),
        _ptr(M1, f32, "M1"), _ptr(M2, f32, "M2"), _ptr(M3, f32, "M3"), _ptr(dO, q.dtype, "dO"),
        *[_ptr(g, f32, "gW") for g in gW], *[_ptr(g, f32, "gM") for g in gM],
        _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dlr"]), _ptr(out["dbeta"]),
        _ptr(out.get("doz")),
        _ptr(out["dW1"]), _ptr(out["dW2"]), _ptr(out["dW3"]), _ptr(out["dM1"]), _ptr(out["dM2"]), _ptr(out["dM3"]),
        ws.data_ptr(), ws.numel(), _stream(stream)))
    return out


# ----------------------------------------------------------------- operators around the layer
# A call's checks depend on its tensors' shapes, strides, types and devices
# and on its parameters alone.  What they yield -- the C structs, the layout
# of results, the workspace size -- is kept for recent combinations, so that a
# serving loop's repeated call costs little beyond its launch.  Nothing of a
# tensor's contents, address or identity is kept.
_PLANS = {}


class _Plan:
    pass


def _meta(t):
    return None if t is None else (t.dtype, t.device, t.shape, t.stride())


def _plan(key, build):
    plan = _PLANS.get(key)
    if plan is None:
        plan = build()
        if len(_PLANS) >= 512:
            _PLANS.clear()
        _PLANS[key] = plan
    return plan


def _int(x, name):
    """A whole number given as any integer type (a tensor of one included):
    its value now, which is what a plan's key has to hold."""
    try:
        n = operator.index(x)
    except TypeError:
        raise ValueError(f"{name} must be a whole number, got {x!r}") from None
    if not -1 << 63 <= n < 1 << 63:
        raise ValueError(f"{name} = {n} is not a 64-bit number")
    return n


def _struct(cls, *values):
    """A C struct of the values, none of which ctypes may have cut to its field's width."""
    s = cls(*values)
    for (name, _), x in zip(cls._fields_, values):
        if isinstance(x, int) and getattr(s, name) != x:
            raise ValueError(f"{name} = {x}: more than the library takes")
    return s


def _one_device(*tensors):
    """The CUDA device that all given tensors share."""
    dev = tensors[0].device
    if dev.type != "cuda":
        raise ValueError("tensors must be on the device")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
    return dev


def _here(index):
    """The raw current stream of the current device, or None if that is not
    device `index`: the short way of a call that names no stream."""
    torch = _torch()
    if torch.cuda.current_device() != index:
        return None
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream().cuda_stream if raw is None else raw(index)


def _on(device, stream, tensors, run):
    """run(handle of the stream) where the call belongs (see _Stream)."""
    if stream is None:
        handle = _here(device.index)
        if handle is not None:
            return run(handle)
    with _Stream(device, stream, tensors) as handle:
        return run(handle)


class _Stream:
    """Where a call runs: with the tensors' device current and, if one is
    given, on `stream` -- what the call allocates then belongs to that stream,
    and the caching allocator learns that the inputs are in use there."""

    def __init__(self, device, stream, tensors):
        torch = _torch()
        self.tensors, self.given, self.guard = tensors, stream, None
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream of {stream.device} for tensors on {device}")
            self.guard = torch.cuda.stream(stream)   # makes its device current too
        elif torch.cuda.current_device() != device.index:
            self.guard = torch.cuda.device(device)
        self.handle = (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)
        if self.given is not None:
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.given)


def _strided(t, name, shape, dtype):
    """Strides of a [batch, heads, tokens, d] tensor with d contiguous."""
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    b, h, l, e = t.stride()
    if e != 1 and shape[3] > 1 and t.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return Strides(b, h, l)


def _lens(t, name, batch):
    if t is not None:
        _check_shapes(**{name: (t, (batch,))})
        _ptr(t, _torch().int64, name)


def _addr(t):
    return None if t is None else t.data_ptr()


def _like(t):
    """The layout of a result like t, in t's order of dimensions where t's rows
    are distinct: a tensor without memory, so that a plan costs none (k and v
    may be a cache that fills the device)."""
    torch = _torch()
    if 0 in t.stride():   # an expanded input: its gradient or result has a place for every element
        return torch.empty(t.shape, dtype=t.dtype, device="meta")
    return torch.empty_like(t, device="meta")


def _new(t, meta):
    """An empty tensor with the shape, strides and type that `meta` recorded, beside t."""
    dtype, _, shape, stride = meta
    if stride == t.stride() and shape == t.shape and dtype == t.dtype:
        return _torch().empty_like(t)   # dense: the recorded strides are what this gives
    return _torch().empty_strided(shape, stride, dtype=dtype, device=t.device)


def _attention_plan(q, k, v, window, sinks, scale, q_lens, k_lens, back):
    torch = _torch()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [batch, heads, tokens, d] and k [batch, kv_heads, tokens, d]")
    (b, h, lq, d), (_, hk, lk, _) = q.shape, k.shape
    plan = _Plan()
    plan.device = _one_device(q, k, v, q_lens, k_lens)
    plan.shape, plan.kshape, plan.dtype = (b, h, lq, d), (b, hk, lk, d), q.dtype
    plan.problem = _struct(Attention, b, h, hk, d, _io_dtype(q), d ** -0.5 if scale is None else scale, lq, lk, window, sinks)
    plan.p = ctypes.byref(plan.problem)
    plan.strides = [_strided(q, "q", plan.shape, q.dtype), _strided(k, "k", plan.kshape, q.dtype),
                    _strided(v, "v", plan.kshape, q.dtype)]
    plan.sq, plan.sk, plan.sv = (ctypes.byref(x) for x in plan.strides)
    _lens(q_lens, "q_lens", b)
    _lens(k_lens, "k_lens", b)
    plan.need = (lib().lact_window_attention_backward_workspace_size if back
                 else lib().lact_window_attention_workspace_size)(plan.p)
    plan.results = [_meta(_like(t)) for t in (q, k, v)]
    plan.rstrides = [Strides(*m[3][:3]) for m in plan.results]
    plan.rq, plan.rk, plan.rv = (ctypes.byref(x) for x in plan.rstrides)
    plan.lse = (torch.float32, None, (b, h, lq), (h * lq, lq, 1))
    return plan


def _attention_back_plan(q, k, v, window, sinks, scale, q_lens, k_lens, o, lse, dO, given):
    plan = _attention_plan(q, k, v, window, sinks, scale, q_lens, k_lens, True)
    _one_device(q, o, lse, dO, *given)
    _check_shapes(lse=(lse, plan.shape[:3]))
    _ptr(lse, _torch().float32, "lse")
    more = [_strided(o, "o", plan.shape, plan.dtype), _strided(dO, "dO", plan.shape, plan.dtype)]
    plan.so, plan.sg = (ctypes.byref(x) for x in more)
    if given[0] is not None:
        more += [_strided(t, f"out[{n}]", s, plan.dtype)
                 for t, n, s in zip(given, ("dq", "dk", "dv"), (plan.shape, plan.kshape, plan.kshape))]
        plan.rq, plan.rk, plan.rv = (ctypes.byref(x) for x in more[2:])
    plan.strides += more
    return plan


def _scratch(need, workspace, device):
    """(address, bytes) of the workspace, and the tensor that holds it."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        ws = _torch().empty(need, dtype=_torch().uint8, device=device)
        return ws.data_ptr(), need, ws
    if workspace.device != device:
        raise ValueError(f"workspace on {workspace.device} for tensors on {device}")
    ws = _workspace(need, workspace, device)
    return ws.data_ptr(), ws.numel(), ws


def window_attention(q, k, v, o=None, *, window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                     q_lens=None, k_lens=None, return_lse: bool = False, lse=None, workspace=None, stream=None):
    """Causal attention over the last `window` keys (0: all) and the first
    `sinks` (lact_window_attention_forward).  q [batch, heads, q_len, d], k, v
    [batch, kv_heads, k_len, d], fp32 or bf16, any strides in multiples of 16
    bytes with d contiguous: token-major tensors come as transposed views.  Row r
    stands at position k_len - q_len + r, with q_lens, k_lens (int64 [batch])
    each sequence's own lengths; scale defaults to d^-1/2.  Returns o in q's
    layout, and with return_lse also lse [batch, heads, q_len] fp32; what is
    allocated here has zeros behind q_lens, given tensors keep what they held."""
    window, sinks, scale = _int(window, "window"), _int(sinks, "sinks"), None if scale is None else float(scale)
    plan = _plan(("attention", window, sinks, scale, _meta(q), _meta(k), _meta(v), _meta(q_lens), _meta(k_lens)),
                 lambda: _attention_plan(q, k, v, window, sinks, scale, q_lens, k_lens, False))
    so = plan.rq
    if o is not None or lse is not None:
        _one_device(q, o, lse)
        if o is not None:
            so = ctypes.byref(_strided(o, "o", plan.shape, plan.dtype))
        _check_shapes(lse=(lse, plan.shape[:3]))
        _ptr(lse, _torch().float32, "lse")

    def run(handle, o=o, lse=lse):
        if o is None:
            o = _new(q, plan.results[0])
            if q_lens is not None:
                o.zero_()
        if lse is None and return_lse:
            lse = _new(q, plan.lse)
            if q_lens is not None:
                lse.zero_()
        ws, ws_bytes, _held = _scratch(plan.need, workspace, q.device)
        st = lib().lact_window_attention_forward(
            plan.p, q.data_ptr(), plan.sq, k.data_ptr(), plan.sk, v.data_ptr(), plan.sv, _addr(q_lens), _addr(k_lens),
            o.data_ptr(), so, _addr(lse), ws, ws_bytes, handle)
        check(st)
        return (o, lse) if return_lse else o

    return _on(plan.device, stream, (q, k, v, o, q_lens, k_lens, lse, workspace), run)


def window_attention_backward(q, k, v, o, lse, *, dO, window: int = 0, sinks: int = 0,
                              scale: Optional[float] = None, q_lens=None, k_lens=None, out=None, workspace=None,
                              stream=None):
    """Backward of window_attention (lact_window_attention_backward): o and lse
    as the forward returned them, dO [batch, heads, q_len, d] in q's dtype.
    Returns a dict of dq, dk, dv in the inputs' dtype and layout, zero behind
    the lengths; `out` (such a dict) is filled instead of allocating."""
    window, sinks, scale = _int(window, "window"), _int(sinks, "sinks"), None if scale is None else float(scale)
    given = (None,) * 3 if out is None else (out["dq"], out["dk"], out["dv"])
    plan = _plan(("attention back", window, sinks, scale, _meta(q), _meta(k), _meta(v), _meta(q_lens), _meta(k_lens),
                  _meta(o), _meta(lse), _meta(dO), _meta(given[0]), _meta(given[1]), _meta(given[2])),
                 lambda: _attention_back_plan(q, k, v, window, sinks, scale, q_lens, k_lens, o, lse, dO, given))

    def run(handle, out=out):
        if out is None:
            m = plan.results
            out = {"dq": _new(q, m[0]), "dk": _new(k, m[1]), "dv": _new(v, m[2])}
        ws, ws_bytes, _held = _scratch(plan.need, workspace, q.device)
        st = lib().lact_window_attention_backward(
            plan.p, q.data_ptr(), plan.sq, k.data_ptr(), plan.sk, v.data_ptr(), plan.sv, _addr(q_lens), _addr(k_lens),
            o.data_ptr(), plan.so, lse.data_ptr(), dO.data_ptr(), plan.sg, out["dq"].data_ptr(), plan.rq,
            out["dk"].data_ptr(), plan.rk, out["dv"].data_ptr(), plan.rv, ws, ws_bytes, handle)
        check(st)
        return out

    return _on(plan.device, stream, (q, k, v, o, lse, dO, q_lens, k_lens, workspace) + given, run)


def _rotary_plan(q, k, freqs, positions, mscale, flags):
    torch = _torch()
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must be [batch, heads, tokens, d]")
    b, h, l, d = q.shape
    if freqs.dim() != 1:
        raise ValueError("freqs must be [pairs]")
    _check_shapes(positions=(positions, (b, l)))
    plan = _Plan()
    plan.device = _one_device(q, k, freqs, positions)
    _ptr(freqs, torch.float64, "freqs")
    _ptr(positions, torch.int64, "positions")
    plan.problem = _struct(RotaryProblem, b, h, 0 if k is None else k.shape[1], d, freqs.shape[0], _io_dtype(q), flags,
                           mscale, l, 0)
    plan.p = ctypes.byref(plan.problem)
    plan.dtype, plan.shape, plan.kshape = q.dtype, (b, h, l, d), None if k is None else (b, k.shape[1], l, d)
    given = [_strided(q, "q", plan.shape, q.dtype)] + ([] if k is None else [_strided(k, "k", plan.kshape, q.dtype)])
    plan.results = [_meta(_like(t)) for t in ((q,) if k is None else (q, k))]
    plan.strides = given + [Strides(*m[3][:3]) for m in plan.results]
    refs = [ctypes.byref(x) for x in plan.strides]
    plan.sq, plan.sk, plan.rq, plan.rk = refs if k is not None else (refs[0], None, refs[1], None)
    return plan


def _rotary(q, k, freqs, positions, start, interleaved, mscale, q_out, k_out, stream, flags):
    start, mscale = _int(start, "start"), float(mscale)
    if interleaved:
        flags |= ROTARY_INTERLEAVED
    plan = _plan(("rotary", _meta(q), _meta(k), _meta(freqs), _meta(positions), mscale, flags),
                 lambda: _rotary_plan(q, k, freqs, positions, mscale, flags))
    p = plan.p
    if positions is None and start:   # another one at every step of a decoding loop: not a part of the plan
        problem = RotaryProblem.from_buffer_copy(plan.problem)
        problem.start, p = start, ctypes.byref(problem)
    rq, rk = plan.rq, plan.rk
    if q_out is not None or k_out is not None:
        _one_device(q, q_out, k_out)
        if q_out is not None:
            rq = ctypes.byref(_strided(q_out, "q_out", plan.shape, plan.dtype))
        if k_out is not None:
            if k is None:
                raise ValueError("k_out is given without k")
            rk = ctypes.byref(_strided(k_out, "k_out", plan.kshape, plan.dtype))

    def run(handle, q_out=q_out, k_out=k_out):
        if q_out is None:
            q_out = _new(q, plan.results[0])
        if k is not None and k_out is None:
            k_out = _new(k, plan.results[1])
        st = lib().lact_rotary(p, q.data_ptr(), plan.sq, _addr(k), plan.sk, freqs.data_ptr(), _addr(positions),
                               q_out.data_ptr(), rq, _addr(k_out), rk, handle)
        check(st)
        return q_out if k is None else (q_out, k_out)

    return _on(plan.device, stream, (q, k, freqs, positions, q_out, k_out), run)


def rotary(q, k=None, *, freqs, positions=None, start: int = 0, interleaved: bool = False, mscale: float = 1.0,
           q_out=None, k_out=None, stream=None):
    """Rotary positions of q [batch, heads, tokens, d] and k [batch, kv_heads,
    tokens, d] in one call (lact_rotary): the first 2 pairs features turn by
    position * freqs (fp64 [pairs] on the device, see rotary_frequencies) and
    are scaled by mscale, the others are copied.  positions int64 [batch,
    tokens], or start + token.  q_out = q and k_out = k work in place.
    Returns q_out, or (q_out, k_out)."""
    return _rotary(q, k, freqs, positions, start, interleaved, mscale, q_out, k_out, stream, 0)


def rotary_backward(dq, dk=None, *, freqs, positions=None, start: int = 0, interleaved: bool = False,
                    mscale: float = 1.0, q_out=None, k_out=None, stream=None):
    """Gradients of rotary's inputs from those of its outputs: the inverse
    turns with the same scale.  Arguments and results as for rotary."""
    return _rotary(dq, dk, freqs, positions, start, interleaved, mscale, q_out, k_out, stream, ROTARY_INVERSE)


def rotary_frequencies(pairs: int, base: float = 10000.0, *, scaling: str = "plain", factor: float = 1.0,
                       context: int = 0, slow: float = 1.0, fast: float = 32.0, device=None):
    """(freqs, mscale) for rotary: base^(-i / pairs), for contexts `factor`
    times the original one scaled "linear", "ntk" or "yarn"
    (lact_rotary_frequencies).  Computed once, kept by the caller."""
    torch = _torch()
    if scaling not in ROTARY_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROTARY_SCALING)}, got {scaling!r}")
    f = torch.empty(max(pairs, 0), dtype=torch.float64)
    m = ctypes.c_float(1.0)
    check(lib().lact_rotary_frequencies(pairs, base, ROTARY_SCALING[scaling], factor, context, slow, fast,
                                        f.data_ptr(), ctypes.byref(m)))
    return f.to("cuda" if device is None else device), m.value


def _rows(t, name, shape, dtype):
    """Row stride of a [..., cols] tensor seen as a matrix."""
    if t is None:
        return 0
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dim() == 2:
        ld, e = t.stride()
        if e != 1 and shape[1] > 1 and t.numel():
            raise ValueError(f"{name}: columns must be contiguous")
        return ld
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (or a matrix with contiguous columns)")
    return shape[-1]


def _norm_plan(x, weight, eps, *others):
    """others: (name, tensor, whether it is in 8 bits)"""
    torch = _torch()
    if x.dim() < 1 or x.shape[-1] == 0:
        raise ValueError("x must be [..., cols] with cols > 0")
    cols = x.shape[-1]
    plan = _Plan()
    plan.device = _one_device(x, weight, *[t for _, t, _ in others])
    _check_shapes(weight=(weight, (cols,)))
    _ptr(weight, torch.float32, "weight")
    plan.problem = _struct(NormProblem, x.numel() // cols, cols, _io_dtype(x), eps)
    plan.p = ctypes.byref(plan.problem)
    plan.shape, plan.cols = tuple(x.shape), cols
    plan.groups = plan.shape[:-1] + ((cols + NORM_GROUP - 1) // NORM_GROUP,)
    plan.ld = [_rows(x, "x", plan.shape, x.dtype)]
    plan.ld += [_rows(t, n, plan.shape, torch.float8_e4m3fn if byte else x.dtype) if t is not None else cols
                for n, t, byte in others]
    plan.need = lib().lact_add_rmsnorm_backward_workspace_size(plan.p)
    return plan


def _stored(x, y, h):
    """Where h is after a forward: in its own tensor, or in x unless y is there."""
    if h is not None:
        return h
    return None if y is not None and y.data_ptr() == x.data_ptr() and x.numel() else x


def add_rmsnorm(x, weight, residual=None, *, eps: float = 1e-6, y=None, h=None, stream=None):
    """h = x + residual and y = h weight / sqrt(mean(h^2) + eps) over the last
    dimension (lact_add_rmsnorm_forward).  x, residual [..., cols] fp32 or
    bf16, weight [cols] fp32.  Returns (y, h); without a residual h is x
    itself, or None where y overwrites it (y = x and no h given).
    h = residual or h = x updates the residual stream in place."""
    eps = float(eps)
    plan = _plan(("norm", eps, _meta(x), _meta(weight), _meta(residual), _meta(y), _meta(h)),
                 lambda: _norm_plan(x, weight, eps, ("residual", residual, False), ("h", h, False), ("y", y, False)))
    ldx, ldr, ldh, ldy = plan.ld

    def run(handle, y=y, h=h):
        if y is None:
            y = x.new_empty(plan.shape)
        if h is None and residual is not None:
            h = x.new_empty(plan.shape)
        st = lib().lact_add_rmsnorm_forward(plan.p, x.data_ptr(), ldx, _addr(residual), ldr, weight.data_ptr(), _addr(h),
                                            ldh, y.data_ptr(), ldy, None, 0, None, handle)
        check(st)
        return y, _stored(x, y, h)

    return _on(plan.device, stream, (x, weight, residual, y, h), run)


def add_rmsnorm_quantised(x, weight, residual=None, *, eps: float = 1e-6, y8=None, scales=None, h=None, y=None,
                          stream=None):
    """As add_rmsnorm, with y in 8-bit floating point: y8 [..., cols]
    float8_e4m3fn and scales [..., ceil(cols / 128)] fp32, so that y is about
    y8 * scale of its group of 128 columns.  Returns (y8, scales, h), h as
    add_rmsnorm returns it; a given y is filled too."""
    torch, eps = _torch(), float(eps)
    plan = _plan(("norm 8", eps, _meta(x), _meta(weight), _meta(residual), _meta(y8), _meta(h), _meta(y)),
                 lambda: _norm_plan(x, weight, eps, ("residual", residual, False), ("h", h, False), ("y", y, False),
                                    ("y8", y8, True)))
    ldx, ldr, ldh, ldy, ld8 = plan.ld
    if scales is not None:
        _one_device(x, scales)
        _check_shapes(scales=(scales, plan.groups))
        _ptr(scales, torch.float32, "scales")

    def run(handle, h=h, y8=y8, scales=scales):
        if y8 is None:
            y8 = x.new_empty(plan.shape, dtype=torch.float8_e4m3fn)
        if scales is None:
            scales = x.new_empty(plan.groups, dtype=torch.float32)
        if h is None and residual is not None:
            h = x.new_empty(plan.shape)
        st = lib().lact_add_rmsnorm_forward(plan.p, x.data_ptr(), ldx, _addr(residual), ldr, weight.data_ptr(), _addr(h),
                                            ldh, _addr(y), ldy, y8.data_ptr(), ld8, scales.data_ptr(), handle)
        check(st)
        return y8, scales, _stored(x, y, h)

    return _on(plan.device, stream, (x, weight, residual, y8, scales, h, y), run)


def add_rmsnorm_backward(h, weight, *, dy, dh=None, eps: float = 1e-6, dx=None, dw=None, workspace=None,
                         stream=None):
    """Backward of add_rmsnorm from the h it returned (lact_add_rmsnorm_backward):
    dy the gradient of y, dh that of h's other use (or None), in h's dtype.
    Returns (dx, dw): dx is the gradient of x and of residual alike, dw [cols]
    fp32 that of the weight."""
    torch, eps = _torch(), float(eps)
    plan = _plan(("norm back", eps, _meta(h), _meta(weight), _meta(dy), _meta(dh), _meta(dx)),
                 lambda: _norm_plan(h, weight, eps, ("dy", dy, False), ("dh", dh, False), ("dx", dx, False)))
    ldh, ldy, lddh, lddx = plan.ld
    if dw is not None:
        _one_device(h, dw)
        _check_shapes(dw=(dw, plan.shape[-1:]))
        _ptr(dw, torch.float32, "dw")

    def run(handle, dx=dx, dw=dw):
        if dx is None:
            dx = h.new_empty(plan.shape)
        if dw is None:
            dw = h.new_empty(plan.cols, dtype=torch.float32)
        ws, ws_bytes, _held = _scratch(plan.need, workspace, h.device)
        st = lib().lact_add_rmsnorm_backward(plan.p, h.data_ptr(), ldh, weight.data_ptr(), dy.data_ptr(), ldy, _addr(dh),
                                             lddh, dx.data_ptr(), lddx, dw.data_ptr(), ws, ws_bytes, handle)
        check(st)
        return dx, dw

    return _on(plan.device, stream, (h, weight, dy, dh, dx, dw, workspace), run)


# ----------------------------------------------------------------- batches of sequences of different lengths
def _strided3(t, name, shape, dtype):
    """Strides of a [heads, tokens, d] tensor with d contiguous."""
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    h, l, e = t.stride()
    if e != 1 and shape[2] > 1 and t.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return Strides(0, h, l)


def _bound(x, name, default, most):
    """A bound that the caller may give on what the device holds."""
    if x is None:
        return default
    x = _int(x, name)
    if x < 0:
        raise ValueError(f"{name} = {x} < 0")
    return min(x, most)


def _packed_rows(plan, q, offsets):
    if q.dim() != 3:
        raise ValueError("q must be [heads, tokens, d]")
    plan.shape, plan.dtype = tuple(q.shape), q.dtype
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be [batch + 1]")
    _ptr(offsets, _torch().int64, "offsets")
    plan.batch = offsets.shape[0] - 1
    plan.lse = (_torch().float32, None, plan.shape[:2], (plan.shape[1], 1))
    plan.strides = [_strided3(q, "q", plan.shape, q.dtype)]


def _packed_plan(q, k, v, offsets, longest, window, sinks, scale):
    if k.dim() != 3:
        raise ValueError("k must be [kv_heads, tokens, d]")
    plan = _Plan()
    plan.device = _one_device(q, k, v, offsets)
    _packed_rows(plan, q, offsets)
    h, t, d = plan.shape
    plan.kshape = (k.shape[0], t, d)
    plan.strides += [_strided3(k, "k", plan.kshape, q.dtype), _strided3(v, "v", plan.kshape, q.dtype)]
    plan.sq, plan.sk, plan.sv = (ctypes.byref(x) for x in plan.strides)
    values = [plan.batch, h, k.shape[0], d, _io_dtype(q), d ** -0.5 if scale is None else scale, t,
              _bound(longest, "longest", t, t), window, sinks]
    plan.problem, plan.clear = _struct(Packed, *values, 0), _struct(Packed, *values, CLEAR_REST)
    plan.p, plan.pc = ctypes.byref(plan.problem), ctypes.byref(plan.clear)
    plan.results = [_meta(_like(x)) for x in (q, k, v)]
    plan.rstrides = [Strides(0, *m[3][:2]) for m in plan.results]
    plan.rq, plan.rk, plan.rv = (ctypes.byref(x) for x in plan.rstrides)
    return plan


def _packed_back_plan(q, k, v, offsets, longest, window, sinks, scale, o, lse, dO, given):
    plan = _packed_plan(q, k, v, offsets, longest, window, sinks, scale)
    _one_device(q, o, lse, dO, *given)
    _check_shapes(lse=(lse, plan.shape[:2]))
    _ptr(lse, _torch().float32, "lse")
    more = [_strided3(o, "o", plan.shape, plan.dtype), _strided3(dO, "dO", plan.shape, plan.dtype)]
    plan.so, plan.sg = (ctypes.byref(x) for x in more)
    if given[0] is not None:
        more += [_strided3(t, f"out[{n}]", s, plan.dtype)
                 for t, n, s in zip(given, ("dq", "dk", "dv"), (plan.shape, plan.kshape, plan.kshape))]
        plan.rq, plan.rk, plan.rv = (ctypes.byref(x) for x in more[2:])
    plan.strides += more
    plan.need = lib().lact_packed_attention_backward_workspace_size(plan.p)
    return plan


def _given_rows(plan, q, o, lse):
    """The strides of o, a given one's or the result's."""
    if o is None and lse is None:
        return plan.rq
    _one_device(q, o, lse)
    _check_shapes(lse=(lse, plan.shape[:2]))
    _ptr(lse, _torch().float32, "lse")
    return plan.rq if o is None else ctypes.byref(_strided3(o, "o", plan.shape, plan.dtype))


def _new_rows(plan, q, o, lse, return_lse):
    """(the problem, o, lse): results to allocate get zeros in rows of no
    sequence, by the call itself where that touches no given tensor."""
    own_o, own_lse = o is None, lse is None and return_lse
    if own_o:
        o = _new(q, plan.results[0])
    given = not own_o or lse is not None
    if own_lse:
        lse = _new(q, plan.lse)
    if given:
        for x, own in ((o, own_o), (lse, own_lse)):
            if own:
                x.zero_()
    return plan.p if given else plan.pc, o, lse


def packed_attention(q, k, v, o=None, *, offsets, longest: Optional[int] = None, window: int = 0, sinks: int = 0,
                     scale: Optional[float] = None, return_lse: bool = False, lse=None, stream=None):
    """Causal attention of sequences packed one after another
    (lact_packed_attention_forward): q [heads, tokens, d], k, v [kv_heads,
    tokens, d], fp32 or bf16, any strides in multiples of 16 bytes with d
    contiguous: token-major tensors come as transposed views.  Sequence b has
    the tokens offsets[b] .. offsets[b + 1] (int64 [batch + 1] on the device),
    `longest` at most (None: it may be all; rows behind are not looked at and
    count as no sequence's).  window, sinks and scale as in
    window_attention.  Returns o in q's layout, and with return_lse also lse
    [heads, tokens] fp32; rows of no sequence are zero in what is allocated
    here and left as they were in given tensors."""
    window, sinks, scale = _int(window, "window"), _int(sinks, "sinks"), None if scale is None else float(scale)
    longest = None if longest is None else _int(longest, "longest")
    plan = _plan(("packed", window, sinks, scale, longest, _meta(q), _meta(k), _meta(v), _meta(offsets)),
                 lambda: _packed_plan(q, k, v, offsets, longest, window, sinks, scale))
    so = _given_rows(plan, q, o, lse)

    def run(handle, o=o, lse=lse):
        p, o, lse = _new_rows(plan, q, o, lse, return_lse)
        check(lib().lact_packed_attention_forward(p, q.data_ptr(), plan.sq, k.data_ptr(), plan.sk, v.data_ptr(), plan.sv,
                                                  offsets.data_ptr(), o.data_ptr(), so, _addr(lse), handle))
        return (o, lse) if return_lse else o

    return _on(plan.device, stream, (q, k, v, offsets, o, lse), run)


def packed_attention_backward(q, k, v, o, lse, *, dO, offsets, longest: Optional[int] = None, window: int = 0,
                              sinks: int = 0, scale: Optional[float] = None, out=None, workspace=None, stream=None):
    """Backward of packed_attention (lact_packed_attention_backward): o and lse
    as the forward returned them, dO [heads, tokens, d] in q's dtype.  Returns a
    dict of dq, dk, dv in the inputs' dtype and layout, zero in rows of no
    sequence; `out` (such a dict) is filled instead of allocating."""
    window, sinks, scale = _int(window, "window"), _int(sinks, "sinks"), None if scale is None else float(scale)
    longest = None if longest is None else _int(longest, "longest")
    given = (None,) * 3 if out is None else (out["dq"], out["dk"], out["dv"])
    plan = _plan(("packed back", window, sinks, scale, longest, _meta(q), _meta(k), _meta(v), _meta(offsets), _meta(o),
                  _meta(lse), _meta(dO), _meta(given[0]), _meta(given[1]), _meta(given[2])),
                 lambda: _packed_back_plan(q, k, v, offsets, longest, window, sinks, scale, o, lse, dO, given))

    def run(handle, out=out):
        if out is None:
            m = plan.results
            out = {"dq": _new(q, m[0]), "dk": _new(k, m[1]), "dv": _new(v, m[2])}
        ws, ws_bytes, _held = _scratch(plan.need, workspace, q.device)
        check(lib().lact_packed_attention_backward(
            plan.p, q.data_ptr(), plan.sq, k.data_ptr(), plan.sk, v.data_ptr(), plan.sv, offsets.data_ptr(), o.data_ptr(),
            plan.so, lse.data_ptr(), dO.data_ptr(), plan.sg, out["dq"].data_ptr(), plan.rq, out["dk"].data_ptr(),
            plan.rk, out["dv"].data_ptr(), plan.rv, ws, ws_bytes, handle))
        return out

    return _on(plan.device, stream, (q, k, v, o, lse, dO, offsets, workspace) + given, run)


def _paged_plan(q, k_pages, v_pages, table, offsets, k_lens, longest, k_len, window, sinks, scale):
    torch = _torch()
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [pages, kv_heads, page, d]")
    plan = _Plan()
    plan.device = _one_device(q, k_pages, v_pages, table, offsets, k_lens)
    _packed_rows(plan, q, offsets)
    h, t, d = plan.shape
    pages, hk, page, _ = k_pages.shape
    pool = (pages, hk, page, d)
    plan.strides += [_strided(k_pages, "k_pages", pool, q.dtype), _strided(v_pages, "v_pages", pool, q.dtype)]
    plan.sq, plan.sk, plan.sv = (ctypes.byref(x) for x in plan.strides)
    _check_shapes(k_lens=(k_lens, (plan.batch,)))
    _ptr(k_lens, torch.int64, "k_lens")
    if table.dim() != 2 or table.shape[0] != plan.batch:
        raise ValueError(f"table has shape {tuple(table.shape)}, expected {(plan.batch, 'width')}")
    _ptr(table, torch.int32, "table")
    width = table.shape[1]
    values = [plan.batch, h, hk, d, _io_dtype(q), d ** -0.5 if scale is None else scale, t,
              _bound(longest, "longest", t, t), _bound(k_len, "k_len", width * page, width * page), window, sinks, pages,
              page, width]
    plan.problem, plan.clear = _struct(Paged, *values, 0), _struct(Paged, *values, CLEAR_REST)
    plan.p, plan.pc = ctypes.byref(plan.problem), ctypes.byref(plan.clear)
    plan.results = [_meta(_like(q))]
    plan.rstrides = Strides(0, *plan.results[0][3][:2])
    plan.rq = ctypes.byref(plan.rstrides)
    plan.need = lib().lact_paged_attention_workspace_size(plan.p)
    return plan


def paged_attention(q, k_pages, v_pages, o=None, *, table, offsets, k_lens, longest: Optional[int] = None,
                    k_len: Optional[int] = None, window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                    return_lse: bool = False, lse=None, workspace=None, stream=None):
    """Attention of new tokens over a paged cache (lact_paged_attention): q
    [heads, tokens, d], of which sequence b has the rows offsets[b] ..
    offsets[b + 1] (int64 [batch + 1]); k_pages, v_pages [pages, kv_heads, page,
    d], page a multiple of 8: token-major pages come as transposed views.
    Sequence b has k_lens[b] keys (int64 [batch]), its new ones among them, in
    the pages table[b] (int32 [batch, width]).  One row a sequence and long
    chunks may be mixed; `longest` and `k_len` bound the rows and keys of a
    sequence (None: all rows, the table's width; rows and keys behind them are
    not looked at, the first ones stand at the end as if they were all) and
    choose how the work is split: chunks of several sequences over a wide table
    are up to two and a half times faster with k_len close to the longest's
    keys.  window, sinks and scale as in window_attention, results as in
    packed_attention."""
    window, sinks, scale = _int(window, "window"), _int(sinks, "sinks"), None if scale is None else float(scale)
    longest = None if longest is None else _int(longest, "longest")
    k_len = None if k_len is None else _int(k_len, "k_len")
    plan = _plan(("paged", window, sinks, scale, longest, k_len, _meta(q), _meta(k_pages), _meta(v_pages), _meta(table),
                  _meta(offsets), _meta(k_lens)),
                 lambda: _paged_plan(q, k_pages, v_pages, table, offsets, k_lens, longest, k_len, window, sinks, scale))
    so = _given_rows(plan, q, o, lse)

    def run(handle, o=o, lse=lse):
        p, o, lse = _new_rows(plan, q, o, lse, return_lse)
        ws, ws_bytes, _held = _scratch(plan.need, workspace, q.device)
        check(lib().lact_paged_attention(p, q.data_ptr(), plan.sq, k_pages.data_ptr(), plan.sk, v_pages.data_ptr(),
                                         plan.sv, offsets.data_ptr(), k_lens.data_ptr(), table.data_ptr(), o.data_ptr(),
                                         so, _addr(lse), ws, ws_bytes, handle))
        return (o, lse) if return_lse else o

    return _on(plan.device, stream, (q, k_pages, v_pages, table, offsets, k_lens, o, lse, workspace), run)


def _slots_plan(lens, counts, table, free, have, page, tokens, given):
    torch = _torch()
    if lens.dim() != 1:
        raise ValueError("lens must be [batch]")
    b = lens.shape[0]
    plan = _Plan()
    plan.device = _one_device(lens, counts, table, free, have, *given.values())
    plan.shapes = {"offsets": (b + 1,), "k_lens": (b,), "slots": (tokens,), "positions": (tokens,), "left": (2,)}
    plan.sizes = [s[0] for s in plan.shapes.values()]
    plan.numbers = sum(plan.sizes)
    _check_shapes(counts=(counts, (b,)), **{n: (t, plan.shapes[n]) for n, t in given.items()})
    if table.dim() != 2 or table.shape[0] != b:
        raise ValueError(f"table has shape {tuple(table.shape)}, expected {(b, 'width')}")
    if free.dim() != 1 or have.dim() != 1 or have.shape[0] not in (1, 2):
        raise ValueError("free must be [entries], free_count [1] or [2]")
    for t, n in [(lens, "lens"), (counts, "counts"), (have, "free_count")] + [(t, n) for n, t in given.items()]:
        _ptr(t, torch.int64, n)
    _ptr(table, torch.int32, "table")
    _ptr(free, torch.int32, "free")
    plan.problem = _struct(Slots, b, page, table.shape[1], free.shape[0], tokens)
    plan.p = ctypes.byref(plan.problem)
    plan.need = lib().lact_page_slots_workspace_size(plan.p)
    return plan


def page_slots(lens, counts, table, free, free_count, *, page: int, tokens: int, out=None, workspace=None, stream=None):
    """Places of a step's new tokens in a paged cache (lact_page_slots).
    Request b holds lens[b] tokens (int64 [batch]) in the pages table[b] (int32
    [batch, width], extended in place) and gets counts[b] more (int64 [batch]),
    in the step's `tokens` rows one request after another.  Pages come off the
    end of free[: free_count] (int32 [entries], int64 [1]; both only read).
    Returns a dict of int64 tensors, what the other operators of a step take:
    offsets [batch + 1] and k_lens [batch] for paged_attention, slots [tokens]
    for page_write, positions [tokens] for rotary, and left [2]: the free pages
    that are left, the next step's free_count, and how many requests got none
    because the pool or their row of the table is full (their slots are -1).
    `out` (such a dict) is filled instead of allocating; its left may be
    free_count itself, of shape [2] (up to 1024 requests, 32768 tokens then
    take 45 us for 8: one workgroup places all rows)."""
    torch, page, tokens = _torch(), _int(page, "page"), _int(tokens, "tokens")
    given = {} if out is None else {n: out[n] for n in ("offsets", "k_lens", "slots", "positions", "left")}
    if tokens < 0:
        raise ValueError(f"tokens = {tokens} < 0")
    plan = _plan(("slots", page, tokens, _meta(lens), _meta(counts), _meta(table), _meta(free), _meta(free_count)) +
                 tuple(_meta(t) for t in given.values()),
                 lambda: _slots_plan(lens, counts, table, free, free_count, page, tokens, given))

    def run(handle, out=out):
        if out is None:   # views of one allocation: five would be half of the call's time
            out = dict(zip(plan.shapes, lens.new_empty(plan.numbers).split_with_sizes(plan.sizes)))
        ws, ws_bytes, _held = _scratch(plan.need, workspace, lens.device)
        check(lib().lact_page_slots(plan.p, lens.data_ptr(), counts.data_ptr(), table.data_ptr(), free.data_ptr(),
                                    free_count.data_ptr(), out["offsets"].data_ptr(), out["k_lens"].data_ptr(),
                                    out["slots"].data_ptr(), out["positions"].data_ptr(), out["left"].data_ptr(), ws,
                                    ws_bytes, handle))
        return out

    return _on(plan.device, stream, (lens, counts, table, free, free_count, workspace) + tuple(given.values()), run)


def _write_plan(k, v, k_pages, v_pages, slots):
    if k.dim() != 3 or k_pages.dim() != 4:
        raise ValueError("k must be [kv_heads, tokens, d] and k_pages [pages, kv_heads, page, d]")
    h, t, d = k.shape
    plan = _Plan()
    plan.device = _one_device(k, v, k_pages, v_pages, slots)
    pool = (k_pages.shape[0], h, k_pages.shape[2], d)
    plan.strides = [_strided3(x, n, (h, t, d), k.dtype) for x, n in ((k, "k"), (v, "v"))]
    plan.strides += [_strided(x, n, pool, k.dtype) for x, n in ((k_pages, "k_pages"), (v_pages, "v_pages"))]
    plan.refs = [ctypes.byref(x) for x in plan.strides]
    _check_shapes(slots=(slots, (t,)))
    _ptr(slots, _torch().int64, "slots")
    plan.problem = _struct(Write, h, d, _io_dtype(k), pool[0], pool[2], t)
    plan.p = ctypes.byref(plan.problem)
    return plan


def page_write(k, v, k_pages, v_pages, *, slots, stream=None):
    """Rows of k and v [kv_heads, tokens, d] into a paged cache
    (lact_page_write): token t goes to slot slots[t] (int64 [tokens], as
    page_slots gives them; -1: nowhere) of k_pages and v_pages [pages, kv_heads,
    page, d], all of one type, any strides in multiples of 16 bytes with d
    contiguous.  Returns (k_pages, v_pages), changed in place."""
    plan = _plan(("write", _meta(k), _meta(v), _meta(k_pages), _meta(v_pages), _meta(slots)),
                 lambda: _write_plan(k, v, k_pages, v_pages, slots))
    a, b, c, d = plan.refs

    def run(handle):
        check(lib().lact_page_write(plan.p, k.data_ptr(), a, v.data_ptr(), b, slots.data_ptr(), k_pages.data_ptr(), c,
                                    v_pages.data_ptr(), d, handle))
        return k_pages, v_pages

    return _on(plan.device, stream, (k, v, k_pages, v_pages, slots), run)


lib()  # fail at import time if the library is missing

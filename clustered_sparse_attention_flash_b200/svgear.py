"""ctypes binding of libsvgear.so (include/svgear.h).

Every function here has the name of a C entry point and only marshals
arguments: torch tensors become device pointers, streams become cudaStream_t
handles.  All arithmetic runs in the CUDA library; there is no fallback.  The
few helpers at the end allocate outputs and workspaces with torch and then call
the same entry points.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
from typing import Dict, Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsvgear.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "svgear.h")

SVGEAR_OK = 0
SVGEAR_ERR_INVALID = -1
SVGEAR_ERR_UNSUPPORTED = -2
SVGEAR_ERR_CUDA = -3
SVGEAR_ERR_TIMEOUT = -4
SVGEAR_ERR_WORKSPACE = -5
SVGEAR_F32 = 0
SVGEAR_BF16 = 1
SVGEAR_ROUTE_ERROR = 0
SVGEAR_ROUTE_MASS = 1
SVGEAR_ROUTE_ERROR_NOV = 2
SVGEAR_BUDGET_ROW = 0
SVGEAR_BUDGET_GLOBAL = 1
SVGEAR_NORM_NONE = 0
SVGEAR_NORM_RMS = 1
SVGEAR_NORM_LAYER = 2
SVGEAR_NORM_CLEAR_REST = 16
SVGEAR_PAIR_ADJACENT = 0
SVGEAR_PAIR_HALF = 1
SVGEAR_QKNORM_NONE = 0
SVGEAR_QKNORM_HEAD = 1
SVGEAR_QKNORM_TOKEN = 2


class SvgearError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({status_string(code)})")
        self.code = code


class svgear_params(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int), ("Nq", ctypes.c_int), ("Nk", ctypes.c_int),
                ("d", ctypes.c_int), ("Cq", ctypes.c_int), ("Ck", ctypes.c_int),
                ("iters", ctypes.c_int), ("rho", ctypes.c_float), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int), ("router", ctypes.c_int), ("budget", ctypes.c_int)]


class svgear_stats(ctypes.Structure):
    _fields_ = [("ms_kmeans_q", ctypes.c_float), ("ms_kmeans_k", ctypes.c_float),
                ("ms_permute", ctypes.c_float), ("ms_block_error", ctypes.c_float),
                ("ms_route", ctypes.c_float), ("ms_attn", ctypes.c_float),
                ("ms_total", ctypes.c_float), ("exec_pairs", ctypes.c_int64),
                ("comp_pairs", ctypes.c_int64), ("ms_attn_kernel", ctypes.c_float)]

    def as_dict(self) -> Dict[str, float]:
        return {k: getattr(self, k) for k, _ in self._fields_}


_VIEW_FIELDS = ["cent_q", "cent_k", "vbar", "labels_q", "labels_k", "counts_q", "counts_k",
                "perm_q", "perm_k", "off_q", "off_k", "Qp", "Kp", "Vp", "key_scalars", "E", "M",
                "mask", "sel", "n_sel", "exec_pairs"]


class svgear_views(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _VIEW_FIELDS]


class svgear_norm_params(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("D", ctypes.c_int), ("G", ctypes.c_int), ("pre", ctypes.c_int),
                ("post", ctypes.c_int), ("eps", ctypes.c_float), ("res_scale", ctypes.c_float),
                ("dtype", ctypes.c_int), ("res_dtype", ctypes.c_int)]


class svgear_rope_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("N", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int),
                ("axes", ctypes.c_int * 3), ("grid", ctypes.c_int * 3), ("origin", ctypes.c_int * 3),
                ("theta", ctypes.c_float * 3), ("pos_scale", ctypes.c_float * 3), ("pairing", ctypes.c_int),
                ("norm", ctypes.c_int), ("eps", ctypes.c_float), ("dtype", ctypes.c_int),
                ("pos_per_batch", ctypes.c_int), ("out_tokens", ctypes.c_int), ("ld", ctypes.c_int64 * 3),
                ("batch", ctypes.c_int64 * 3), ("grad_ld", ctypes.c_int64), ("grad_batch", ctypes.c_int64)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_PP = ctypes.POINTER(svgear_params)
_NP = ctypes.POINTER(svgear_norm_params)
_RP = ctypes.POINTER(svgear_rope_params)

_SIGS = {
    "svgear_version": (ctypes.c_char_p, []),
    "svgear_status_string": (ctypes.c_char_p, [_I]),
    "svgear_launch_count": (ctypes.c_longlong, []),
    "svgear_get_status": (_I, [_P]),
    "svgear_selftest_wait": (_I, [ctypes.c_longlong, _P]),
    "svgear_kmeans_workspace_size": (_SZ, [_I, _I, _I, _I]),
    "svgear_kmeans": (_I, [_P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "svgear_permute_workspace_size": (_SZ, [_I, _I, _I]),
    "svgear_permute": (_I, [_P, _I, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "svgear_block_error_workspace_size": (_SZ, [_PP]),
    "svgear_block_error": (_I, [_P, _P, _P, _P, _P, _P, _P, _PP, _P, _P, _P, _SZ, _P]),
    "svgear_block_error_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _P, _PP, _P, _P, _P]),
    "svgear_route": (_I, [_P, _P, _P, _PP, _P, _P, _P, _P, _P]),
    "svgear_route_global": (_I, [_P, _P, _P, _P, _PP, _P, _P, _P, _P, _P]),
    "svgear_hybrid_attn_workspace_size": (_SZ, [_PP]),
    "svgear_hybrid_attn": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _PP, _P, _P, _SZ, _P]),
    "svgear_workspace_size": (_SZ, [_PP]),
    "svgear_forward_views": (_I, [_PP, _P, _SZ, ctypes.POINTER(svgear_views)]),
    "svgear_forward": (_I, [_P, _P, _P, _PP, _P, _P, _P, _P, _SZ, _P, ctypes.POINTER(svgear_stats)]),
    "svgear_block_norm": (_I, [_P] * 9 + [_NP, _P, _P, _P]),
    "svgear_block_norm_backward_workspace_size": (_SZ, [_NP]),
    "svgear_block_norm_backward": (_I, [_P] * 10 + [_NP] + [_P] * 9 + [_SZ, _P]),
    "svgear_qkv_rope": (_I, [_P] * 6 + [_RP] + [_P] * 4),
    "svgear_qkv_rope_backward_workspace_size": (_SZ, [_RP]),
    "svgear_qkv_rope_backward": (_I, [_P] * 8 + [_RP] + [_P] * 6 + [_SZ, _P]),
    "svgear_mx_quantize": (_I, [_P, _I, _I, _I, _I, _P, _P, _P]),
    "svgear_mx_dequantize": (_I, [_P, _P, _I, _I, _P, _I, _P]),
    "svgear_mx_product": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
}

_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if libsvgear.so has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libsvgear.so not found at {LIB_PATH}; run "
                              "`python -m clustered_sparse_attention_flash_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def header_functions():
    """Names of the entry points declared in include/svgear.h."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"SVGEAR_API\s+[\w\s\*]*?\b(svgear_\w+)\s*\(", txt)))


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_cuda:
            raise ValueError("device tensor expected")
        if not x.is_contiguous():
            raise ValueError("contiguous tensor expected")
        return x.data_ptr()
    raise TypeError(f"cannot pass {type(x)} as a pointer")


def _rows_ptr(x) -> Optional[int]:
    """Pointer of a tensor whose strides travel in the parameter block."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("device tensor expected")
    return x.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(fn: str, code: int) -> None:
    if code != SVGEAR_OK:
        raise SvgearError(fn, code)


def _fits(fn: str, *counts: int) -> None:
    """Refuses counts that a C int does not hold: ctypes would cut them to 32 bits, and a call of fewer rows run."""
    if max(counts) > 0x7fffffff:
        raise SvgearError(fn, SVGEAR_ERR_UNSUPPORTED)


def params(H, Nq, Nk, d, Cq, Ck, iters, rho, scale=0.0, dtype=SVGEAR_BF16,
           router=SVGEAR_ROUTE_ERROR, budget=SVGEAR_BUDGET_ROW) -> svgear_params:
    return svgear_params(H, Nq, Nk, d, Cq, Ck, iters, rho, scale, dtype, router, budget)


# ----------------------------------------------------------------- entries

def svgear_version() -> str:
    return lib().svgear_version().decode()


def svgear_launch_count() -> int:
    return int(lib().svgear_launch_count())


def status_string(code: int) -> str:
    return lib().svgear_status_string(code).decode()


svgear_status_string = status_string


def svgear_get_status(stream=None) -> int:
    return lib().svgear_get_status(_stream(stream))


def svgear_selftest_wait(limit_ns: int, stream=None) -> None:
    _check("svgear_selftest_wait", lib().svgear_selftest_wait(int(limit_ns), _stream(stream)))


def svgear_kmeans_workspace_size(H, N, d, C) -> int:
    return lib().svgear_kmeans_workspace_size(H, N, d, C)


def svgear_kmeans(X, dtype, H, N, d, C, iters, init, cent, labels, counts, ws, ws_bytes, stream=None):
    _check("svgear_kmeans", lib().svgear_kmeans(
        _ptr(X), dtype, H, N, d, C, iters, _ptr(init), _ptr(cent), _ptr(labels), _ptr(counts),
        _ptr(ws), ws_bytes, _stream(stream)))


def svgear_permute_workspace_size(H, N, C) -> int:
    return lib().svgear_permute_workspace_size(H, N, C)


def svgear_permute(X, dtype, labels, H, N, d, C, Xp, perm, offsets, V, Vp, Vbar, key_scalars,
                   ws, ws_bytes, stream=None):
    _check("svgear_permute", lib().svgear_permute(
        _ptr(X), dtype, _ptr(labels), H, N, d, C, _ptr(Xp), _ptr(perm), _ptr(offsets), _ptr(V),
        _ptr(Vp), _ptr(Vbar), _ptr(key_scalars), _ptr(ws), ws_bytes, _stream(stream)))


def svgear_block_error_workspace_size(p: svgear_params) -> int:
    return lib().svgear_block_error_workspace_size(ctypes.byref(p))


def svgear_block_error(Qbar, Kbar, Vbar, Kp, Vp, k_off, key_scalars, p, E, M, ws, ws_bytes,
                       stream=None):
    _check("svgear_block_error", lib().svgear_block_error(
        _ptr(Qbar), _ptr(Kbar), _ptr(Vbar), _ptr(Kp), _ptr(Vp), _ptr(k_off), _ptr(key_scalars),
        ctypes.byref(p), _ptr(E), _ptr(M), _ptr(ws), ws_bytes, _stream(stream)))


def svgear_block_error_noalloc(Qbar, Kbar, Vbar, Kp, Vp, k_off, key_scalars, p, E, M, stream=None):
    _check("svgear_block_error_noalloc", lib().svgear_block_error_noalloc(
        _ptr(Qbar), _ptr(Kbar), _ptr(Vbar), _ptr(Kp), _ptr(Vp), _ptr(k_off), _ptr(key_scalars),
        ctypes.byref(p), _ptr(E), _ptr(M), _stream(stream)))


def svgear_route(E, k_counts, q_counts, p, mask, sel, n_sel, exec_pairs, stream=None):
    _check("svgear_route", lib().svgear_route(
        _ptr(E), _ptr(k_counts), _ptr(q_counts), ctypes.byref(p), _ptr(mask), _ptr(sel),
        _ptr(n_sel), _ptr(exec_pairs), _stream(stream)))


def svgear_route_global(E, M, k_counts, q_counts, p, mask, sel, n_sel, exec_pairs, stream=None):
    _check("svgear_route_global", lib().svgear_route_global(
        _ptr(E), _ptr(M), _ptr(k_counts), _ptr(q_counts), ctypes.byref(p), _ptr(mask), _ptr(sel),
        _ptr(n_sel), _ptr(exec_pairs), _stream(stream)))


def svgear_hybrid_attn_workspace_size(p: svgear_params) -> int:
    return lib().svgear_hybrid_attn_workspace_size(ctypes.byref(p))


def svgear_hybrid_attn(Qp, Kp, Vp, q_off, k_off, perm_q, Kbar, Vbar, sel, n_sel, p, O, ws,
                       ws_bytes, stream=None):
    _check("svgear_hybrid_attn", lib().svgear_hybrid_attn(
        _ptr(Qp), _ptr(Kp), _ptr(Vp), _ptr(q_off), _ptr(k_off), _ptr(perm_q), _ptr(Kbar),
        _ptr(Vbar), _ptr(sel), _ptr(n_sel), ctypes.byref(p), _ptr(O), _ptr(ws), ws_bytes,
        _stream(stream)))


def svgear_workspace_size(p: svgear_params) -> int:
    return lib().svgear_workspace_size(ctypes.byref(p))


def svgear_forward_views(p: svgear_params, ws, ws_bytes) -> svgear_views:
    v = svgear_views()
    _check("svgear_forward_views", lib().svgear_forward_views(
        ctypes.byref(p), _ptr(ws), ws_bytes, ctypes.byref(v)))
    return v


def svgear_forward(Q, K, V, p, init_q, init_k, O, ws, ws_bytes, stream=None, stats=None):
    _check("svgear_forward", lib().svgear_forward(
        _ptr(Q), _ptr(K), _ptr(V), ctypes.byref(p), _ptr(init_q), _ptr(init_k), _ptr(O),
        _ptr(ws), ws_bytes, _stream(stream), ctypes.byref(stats) if stats is not None else None))


def svgear_block_norm(x, y, gate, scale, shift, weight, bias, post_weight, offsets, p, r, h, stream=None):
    _check("svgear_block_norm", lib().svgear_block_norm(
        _ptr(x), _ptr(y), _ptr(gate), _ptr(scale), _ptr(shift), _ptr(weight), _ptr(bias), _ptr(post_weight),
        _ptr(offsets), ctypes.byref(p), _ptr(r), _ptr(h), _stream(stream)))


def svgear_block_norm_backward_workspace_size(p: svgear_norm_params) -> int:
    return lib().svgear_block_norm_backward_workspace_size(ctypes.byref(p))


def svgear_block_norm_backward(x, y, dr, dh, gate, scale, weight, bias, post_weight, offsets, p, dx, dy, dgate,
                               dscale, dshift, dweight, dbias, dpost_weight, ws, ws_bytes, stream=None):
    _check("svgear_block_norm_backward", lib().svgear_block_norm_backward(
        _ptr(x), _ptr(y), _ptr(dr), _ptr(dh), _ptr(gate), _ptr(scale), _ptr(weight), _ptr(bias),
        _ptr(post_weight), _ptr(offsets), ctypes.byref(p), _ptr(dx), _ptr(dy), _ptr(dgate), _ptr(dscale),
        _ptr(dshift), _ptr(dweight), _ptr(dbias), _ptr(dpost_weight), _ptr(ws), ws_bytes, _stream(stream)))


def svgear_qkv_rope(q, k, v, wq, wk, positions, p, Q, K, V, stream=None):
    """q, k, v may be strided rows (p.ld, p.batch); the outputs may be head-major views (p.out_tokens)."""
    _check("svgear_qkv_rope", lib().svgear_qkv_rope(
        _rows_ptr(q), _rows_ptr(k), _rows_ptr(v), _ptr(wq), _ptr(wk), _ptr(positions), ctypes.byref(p),
        _rows_ptr(Q), _rows_ptr(K), _rows_ptr(V), _stream(stream)))


def svgear_qkv_rope_backward_workspace_size(p: svgear_rope_params) -> int:
    return lib().svgear_qkv_rope_backward_workspace_size(ctypes.byref(p))


def svgear_qkv_rope_backward(dQ, dK, dV, q, k, wq, wk, positions, p, dq, dk, dv, dwq, dwk, ws, ws_bytes,
                             stream=None):
    _check("svgear_qkv_rope_backward", lib().svgear_qkv_rope_backward(
        _rows_ptr(dQ), _rows_ptr(dK), _rows_ptr(dV), _rows_ptr(q), _rows_ptr(k), _ptr(wq), _ptr(wk),
        _ptr(positions), ctypes.byref(p), _rows_ptr(dq), _rows_ptr(dk), _rows_ptr(dv), _ptr(dwq), _ptr(dwk),
        _ptr(ws), ws_bytes, _stream(stream)))


def svgear_mx_quantize(X, dtype, M, K, head_d, codes, scales, stream=None):
    _fits("svgear_mx_quantize", M, K, head_d)
    _check("svgear_mx_quantize", lib().svgear_mx_quantize(
        _ptr(X), dtype, M, K, head_d, _ptr(codes), _ptr(scales), _stream(stream)))


def svgear_mx_dequantize(codes, scales, M, K, Y, dtype, stream=None):
    _fits("svgear_mx_dequantize", M, K)
    _check("svgear_mx_dequantize", lib().svgear_mx_dequantize(
        _ptr(codes), _ptr(scales), M, K, _ptr(Y), dtype, _stream(stream)))


def svgear_mx_product(a_codes, a_scales, w_codes, w_scales, bias, M, N, K, Y, stream=None):
    _fits("svgear_mx_product", M, N, K)
    _check("svgear_mx_product", lib().svgear_mx_product(
        _ptr(a_codes), _ptr(a_scales), _ptr(w_codes), _ptr(w_scales), _ptr(bias), M, N, K, _ptr(Y),
        _stream(stream)))


# ------------------------------------------------------- torch conveniences

def dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return SVGEAR_BF16
    if t.dtype == torch.float32:
        return SVGEAR_F32
    raise ValueError(f"unsupported dtype {t.dtype}")


def workspace(nbytes: int, device="cuda"):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def view_tensors(p: svgear_params, ws) -> Dict[str, "object"]:
    """torch tensors aliasing the intermediates svgear_forward leaves in `ws`."""
    import torch
    v = svgear_forward_views(p, ws, ws.numel())
    H, Nq, Nk, d, Cq, Ck = p.H, p.Nq, p.Nk, p.d, p.Cq, p.Ck
    tdt = torch.bfloat16 if p.dtype == SVGEAR_BF16 else torch.float32
    es = 2 if p.dtype == SVGEAR_BF16 else 4
    base = ws.data_ptr()
    spec = {
        "cent_q": (torch.float32, (H, Cq, d)), "cent_k": (torch.float32, (H, Ck, d)),
        "vbar": (torch.float32, (H, Ck, d)), "labels_q": (torch.int32, (H, Nq)),
        "labels_k": (torch.int32, (H, Nk)), "counts_q": (torch.int32, (H, Cq)),
        "counts_k": (torch.int32, (H, Ck)), "perm_q": (torch.int32, (H, Nq)),
        "perm_k": (torch.int32, (H, Nk)), "off_q": (torch.int32, (H, Cq + 1)),
        "off_k": (torch.int32, (H, Ck + 1)), "Qp": (tdt, (H, Nq, d)), "Kp": (tdt, (H, Nk, d)),
        "Vp": (tdt, (H, Nk, d)), "key_scalars": (torch.float32, (3, H, Nk)),
        "E": (torch.float32, (H, Cq, Ck)), "M": (torch.float32, (H, Cq)),
        "mask": (torch.uint8, (H, Cq, Ck)), "sel": (torch.int32, (H, Cq, Ck)),
        "n_sel": (torch.int32, (H, Cq)), "exec_pairs": (torch.int64, (H,)),
    }
    out = {}
    for name, (dt, shape) in spec.items():
        off = getattr(v, name) - base
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        out[name] = ws[off:off + nbytes].view(dt).view(shape)
    del es
    return out


def forward(Q, K, V, Cq: int, Ck: int, iters: int, rho: float, scale: float = 0.0,
            init_q=None, init_k=None, ws=None, stream=None, stats: bool = False,
            router: int = SVGEAR_ROUTE_ERROR, budget: int = SVGEAR_BUDGET_ROW):
    """Allocate O (and the workspace unless given) and run svgear_forward.
    Returns (O, ws, params, stats-dict or None)."""
    import torch
    H, Nq, d = Q.shape
    Nk = K.shape[1]
    p = params(H, Nq, Nk, d, Cq, Ck, iters, rho, scale, dtype_code(Q), router, budget)
    need = svgear_workspace_size(p)
    if need == 0:
        raise SvgearError("svgear_workspace_size", SVGEAR_ERR_INVALID)
    if ws is None or ws.numel() < need:
        ws = workspace(need, Q.device)
    O = torch.empty_like(Q)
    st = svgear_stats() if stats else None
    svgear_forward(Q, K, V, p, init_q, init_k, O, ws, ws.numel(), stream, st)
    return O, ws, p, (st.as_dict() if st is not None else None)


# ---- around the attention: norms, rotary positions, 4-bit projections
#
# These helpers run on the device their tensors are on, whatever device is
# current, and on `stream` (default: that device's current stream).  Outputs
# and workspaces are allocated on the same stream, so the caching allocator
# never hands their memory to work the kernels are not ordered with.  They
# check every tensor themselves and call the library with plain pointers: on
# small inputs the host's time is the call's time.  They do not take part in
# autograd: their results are detached, and a gradient is a call of its own
# (block_norm_backward, qkv_rope_backward).


class _On:
    """Makes `device` current, and `stream` its current stream when one is given; enters as the stream's handle."""
    __slots__ = ("device", "ctx")

    def __init__(self, device, stream):
        import torch
        self.device = device.index
        self.ctx = None
        if self.device != torch.cuda.current_device():
            self.ctx = [torch.cuda.device(device)]
        if stream is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
            elif stream.device.index != self.device:  # entering it would make its device current
                raise ValueError(f"stream: one of {device} expected, got one of {stream.device}")
            self.ctx = (self.ctx or []) + [torch.cuda.stream(stream)]

    def __enter__(self):
        import torch
        if self.ctx:
            for c in self.ctx:
                c.__enter__()
        return torch._C._cuda_getCurrentRawStream(self.device)

    def __exit__(self, *e):
        if self.ctx:
            for c in reversed(self.ctx):
                c.__exit__(*e)


def _want(name, t, dtype, shape, device, contiguous=True):
    """Checks one optional tensor argument against what the call expects; returns its address."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or t.shape != shape or (contiguous and not t.is_contiguous()):
        if t.device != device:
            raise ValueError(f"{name}: a tensor on {device} expected, got {t.device}")
        if t.dtype is not dtype:
            raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
        raise ValueError(f"{name}: contiguous tensor expected")
    return t.data_ptr()


def _code(dtype) -> int:
    import torch
    if dtype is torch.bfloat16:
        return SVGEAR_BF16
    if dtype is torch.float32:
        return SVGEAR_F32
    raise ValueError(f"unsupported dtype {dtype}")


def _norm_call(x, y, dtype, gate, scale, shift, weight, bias, post_weight, pre, post, eps, res_scale, offsets):
    """Checks the inputs shared by forward and backward; returns the parameter block and the addresses of
    x, y, gate, scale, shift, weight, bias, post_weight and offsets."""
    import torch
    if x.dim() != 2:
        raise ValueError(f"x: [N, D] expected, got shape {tuple(x.shape)}")
    if not x.is_cuda:
        raise ValueError("x: device tensor expected")
    if not x.is_contiguous():
        raise ValueError("x: contiguous tensor expected")
    N, D = x.shape
    dev, f32 = x.device, torch.float32
    G = 1
    if offsets is not None:
        if offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError("offsets: [G + 1] int32 expected")
        G = offsets.shape[0] - 1
    elif gate is not None:
        G = gate.shape[0]
    elif scale is not None:
        G = scale.shape[0]
    elif shift is not None:
        G = shift.shape[0]
    _fits("svgear_block_norm", N, D, G)
    p = svgear_norm_params(N, D, G, pre, post, eps, res_scale, _code(dtype), _code(x.dtype))
    return p, (x.data_ptr(), _want("y", y, dtype, (N, D), dev), _want("gate", gate, f32, (G, D), dev),
               _want("scale", scale, f32, (G, D), dev), _want("shift", shift, f32, (G, D), dev),
               _want("weight", weight, f32, (D,), dev), _want("bias", bias, f32, (D,), dev),
               _want("post_weight", post_weight, f32, (D,), dev), _want("offsets", offsets, torch.int32, (G + 1,), dev))


def block_norm(x, y=None, *, gate=None, scale=None, shift=None, weight=None, bias=None, post_weight=None,
               pre: int = SVGEAR_NORM_LAYER, post: int = SVGEAR_NORM_NONE, eps: float = 1e-6,
               res_scale: float = 1.0, offsets=None, dtype=None, want_h: bool = True, stream=None):
    """r = res_scale x + gate P(y) post_weight and h = (Q(r) weight + bias)(1 + scale) + shift through
    svgear_block_norm.  x [N, D], y [N, D] or None (r is x); gate, scale, shift [G, D] with the groups given
    by offsets [G+1] or N/G rows each.  h has y's type, or `dtype` (default x's) without y.  Rows from
    offsets[G] on belong to no group and are zero in r and h (without y, r is x as it is).
    Returns (r, h); h is None with want_h=False."""
    import torch
    if y is not None and dtype is not None and dtype != y.dtype:
        raise ValueError(f"dtype {dtype} differs from y's {y.dtype}")
    dtype = y.dtype if y is not None else dtype or x.dtype
    p, ptrs = _norm_call(x, y, dtype, gate, scale, shift, weight, bias, post_weight, pre, post, eps, res_scale, offsets)
    if offsets is not None:
        p.pre |= SVGEAR_NORM_CLEAR_REST
    with _On(x.device, stream) as st:
        r = torch.empty_like(x) if y is not None else None
        h = torch.empty_like(x, dtype=dtype) if want_h else None
        _check("svgear_block_norm", lib().svgear_block_norm(
            *ptrs, ctypes.byref(p), None if r is None else r.data_ptr(), None if h is None else h.data_ptr(), st))
    return (x if r is None else r), h


def block_norm_backward(x, y, dr, dh, *, gate=None, scale=None, shift=None, weight=None, bias=None,
                        post_weight=None, pre: int = SVGEAR_NORM_LAYER, post: int = SVGEAR_NORM_NONE,
                        eps: float = 1e-6, res_scale: float = 1.0, offsets=None, stream=None):
    """Gradients of block_norm for the gradients dr of r and dh of h (one may be None), through
    svgear_block_norm_backward.  The other arguments are the forward's.  Returns a dict with dx, dy, dgate,
    dscale, dshift, dweight, dbias and dpost_weight; None for what the forward was not given.  Rows from
    offsets[G] on add to no sum and are zero in dx and dy (without y, where r is x, dx is dr there)."""
    import torch
    if dr is None and dh is None:
        raise ValueError("dr or dh expected")
    dtype = y.dtype if y is not None else dh.dtype if dh is not None else x.dtype
    p, ptrs = _norm_call(x, y, dtype, gate, scale, shift, weight, bias, post_weight, pre, post, eps, res_scale, offsets)
    px, py, pgate, pscale, _, pweight, pbias, ppost, poff = ptrs
    if offsets is not None:
        p.pre |= SVGEAR_NORM_CLEAR_REST
    pdr, pdh = _want("dr", dr, x.dtype, x.shape, x.device), _want("dh", dh, dtype, x.shape, x.device)
    with _On(x.device, stream) as st:
        given = {"dx": x, "dy": y, "dgate": gate, "dscale": scale, "dshift": shift, "dweight": weight, "dbias": bias,
                 "dpost_weight": post_weight}
        out = {n: None if t is None else torch.empty_like(t) for n, t in given.items()}
        need = svgear_block_norm_backward_workspace_size(p)
        ws = workspace(need, x.device)
        _check("svgear_block_norm_backward", lib().svgear_block_norm_backward(
            px, py, pdr, pdh, pgate, pscale, pweight, pbias, ppost, poff, ctypes.byref(p),
            *(None if t is None else t.data_ptr() for t in out.values()), ws.data_ptr(), ws.numel(), st))
    return out


_ROPE_FMT = struct.Struct("4i9i6f2if3i8q")  # svgear_rope_params, natively aligned


def _three(v):
    return tuple(v) if isinstance(v, (tuple, list)) else (v, v, v)


def rope_params(B, N, H, d, axes, grid=(0, 0, 0), origin=0, theta=10000.0, pos_scale=1.0,
                pairing: int = SVGEAR_PAIR_ADJACENT, norm: int = SVGEAR_QKNORM_NONE, eps: float = 1e-6,
                dtype: int = SVGEAR_BF16, pos_per_batch: int = 0, out_tokens: int = 0, ld=None, batch=None,
                grad_ld=None, grad_batch=None) -> svgear_rope_params:
    """Parameter block; origin, theta and pos_scale are one value or one per axis, ld and batch the strides of
    q, k and v (default: dense rows [B, N, H, d], as for the gradients)."""
    if len(axes) != 3 or len(grid) != 3:
        raise ValueError("axes and grid have three entries: time, height, width")
    row, entry = H * d, N * H * d
    return svgear_rope_params.from_buffer_copy(_ROPE_FMT.pack(
        B, N, H, d, *axes, *grid, *_three(origin), *_three(theta), *_three(pos_scale), pairing, norm, eps, dtype,
        pos_per_batch, out_tokens, *(ld or (row, row, row)), *(batch or (entry, entry, entry)),
        row if grad_ld is None else grad_ld, entry if grad_batch is None else grad_batch))


def _rope_call(rows, wq, wk, axes, grid, positions, origin, theta, pos_scale, pairing, norm, eps, shape, dev, dtype,
               out_tokens, grad_ld=None, grad_batch=None):
    """Checks [B, N, H, d] or [N, H, d] rows, weights and positions; returns the parameter block and the
    addresses of the rows, of wq, wk and of positions."""
    import torch
    code = _code(dtype)
    if len(shape) not in (3, 4):
        raise ValueError(f"rows [B, N, H, d] or [N, H, d] expected, got shape {tuple(shape)}")
    B, (N, H, d) = (shape[0] if len(shape) == 4 else 1), shape[-3:]
    ld, batch, ptrs = [H * d] * 3, [N * H * d] * 3, [None] * 3
    for i, t in enumerate(rows):
        if t is None:
            continue
        ptrs[i] = _want("qkv"[i], t, dtype, shape, dev, contiguous=False)
        st = t.stride()
        if st[-1] != 1 or (H > 1 and st[-2] != d):
            raise ValueError(f"{'qkv'[i]}: the heads of a token have to be dense")
        if N > 1:
            ld[i] = st[-3]
        if B > 1:
            batch[i] = st[0]
    per_batch = int(positions is not None and positions.dim() == 3)
    cols = (d if norm == SVGEAR_QKNORM_HEAD else H * d,)
    ptrs += [_want("wq", wq, torch.float32, cols, dev), _want("wk", wk, torch.float32, cols, dev),
             _want("positions", positions, torch.int32, (B, N, 3) if per_batch else (N, 3), dev)]
    return rope_params(B, N, H, d, axes, grid or (0, 0, 0), origin, theta, pos_scale, pairing, norm, eps, code,
                       per_batch, out_tokens, ld, batch, grad_ld, grad_batch), ptrs


def qkv_rope(q, k, v, *, axes, grid=None, positions=None, wq=None, wk=None, origin=0, theta=10000.0, pos_scale=1.0,
             pairing: int = SVGEAR_PAIR_ADJACENT, norm: int = SVGEAR_QKNORM_NONE, eps: float = 1e-6, out=None,
             out_at: int = 0, stream=None):
    """Q, K, V [B*H, N, d] for the attention from projection rows [B, N, H, d] or [N, H, d] (views of a fused
    projection may be passed), through svgear_qkv_rope: RMS norm of q and k, rotary positions on three axes,
    head-major order.  Each of q, k, v may be None.  With out=(Q, K, V), tensors [B*H, M, d], the tokens go to
    rows [out_at, out_at + N) and the others stay (a joint sequence, part by part).  Returns (Q, K, V)."""
    import torch
    x = q if q is not None else k if k is not None else v
    if x is None:
        raise ValueError("one of q, k, v expected")
    if out is not None and (len(out) != 3 or any((o is None) != (t is None) or (o is not None and o.dim() != 3)
                                                 for o, t in zip(out, (q, k, v)))):
        raise ValueError("out: [B*H, M, d] for each of q, k, v that is given, None for the others")
    if not x.is_cuda:
        raise ValueError("device tensor expected")
    dev, dtype, shape = x.device, x.dtype, x.shape
    N = shape[-3] if len(shape) >= 3 else 0
    M = N if out is None else next(t.shape[1] for t in out if t is not None)
    p, ptrs = _rope_call((q, k, v), wq, wk, axes, grid, positions, origin, theta, pos_scale, pairing, norm, eps, shape,
                         dev, dtype, M)
    shape = (p.B * p.H, M, p.d)
    if not 0 <= out_at <= M - N:
        raise ValueError(f"out_at {out_at}: {N} tokens do not fit into {M} rows there")
    with _On(dev, stream) as st:
        if out is None:
            out = tuple([None if t is None else torch.empty(shape, dtype=dtype, device=dev) for t in (q, k, v)])
            dst = [None if t is None else t.data_ptr() for t in out]
        else:
            at = out_at * p.d * x.element_size()
            dst = [None if t is None else _want(n, t, dtype, shape, dev) + at for n, t in zip("QKV", out)]
        _check("svgear_qkv_rope", lib().svgear_qkv_rope(*ptrs, ctypes.byref(p), *dst, st))
    return tuple(out)


def qkv_rope_backward(dQ, dK, dV, q=None, k=None, *, axes, grid=None, positions=None, wq=None, wk=None, origin=0,
                      theta=10000.0, pos_scale=1.0, pairing: int = SVGEAR_PAIR_ADJACENT,
                      norm: int = SVGEAR_QKNORM_NONE, eps: float = 1e-6, H: Optional[int] = None, stream=None):
    """Gradients of qkv_rope for the gradients of Q, K, V ([B*H, N, d], each may be None), through
    svgear_qkv_rope_backward.  q and k are the forward's inputs; without them (no norm) H gives the heads.
    dq, dk and dv are views [B, N, H, d] of one fused buffer [B, N, 3, H, d] ([N, H, d] when q or k has no
    batch).  Returns a dict with dq, dk, dv, dwq, dwk; None for what was not given."""
    import torch
    grads = (dQ, dK, dV)
    have = [i for i in range(3) if grads[i] is not None]
    if not have:
        raise ValueError("one of dQ, dK, dV expected")
    g = grads[have[0]]
    if not g.is_cuda or g.dim() != 3:
        raise ValueError("gradients [B*H, N, d] on a device expected")
    ref = q if q is not None else k
    if ref is not None:
        shape = ref.shape
    else:
        if not H or g.shape[0] % H:
            raise ValueError("H: the number of heads expected where q and k are not given")
        shape = (g.shape[0] // H, g.shape[1], H, g.shape[2])
    if norm != SVGEAR_QKNORM_NONE and ((dQ is not None and q is None) or (dK is not None and k is None)):
        raise ValueError("q and k expected with a norm")
    width = shape[-2] * shape[-1] if len(shape) >= 3 else 0
    p, (pq, pk, _, pwq, pwk, ppos) = _rope_call(
        (q, k, None), wq, wk, axes, grid, positions, origin, theta, pos_scale, pairing, norm, eps, shape, g.device, g.dtype,
        0, len(have) * width, len(have) * width * shape[-3] if len(shape) >= 3 else 0)
    ptrs = [_want(n, t, g.dtype, (p.B * p.H, p.N, p.d), g.device) for n, t in zip(("dQ", "dK", "dV"), grads)]
    with _On(g.device, stream) as st:
        fused = torch.empty((p.B, p.N, len(have), p.H, p.d), dtype=g.dtype, device=g.device)
        rows, dst = [None] * 3, [None] * 3
        for at, i in enumerate(have):
            rows[i] = fused[:, :, at] if len(shape) == 4 else fused[0, :, at]
            dst[i] = fused.data_ptr() + at * width * fused.element_size()
        dwq = torch.empty_like(wq) if wq is not None and dQ is not None else None
        dwk = torch.empty_like(wk) if wk is not None and dK is not None else None
        ws, need = None, 0
        if dwq is not None or dwk is not None:
            need = svgear_qkv_rope_backward_workspace_size(p)
            ws = workspace(need, g.device)
        _check("svgear_qkv_rope_backward", lib().svgear_qkv_rope_backward(
            *ptrs, pq, pk, pwq, pwk, ppos, ctypes.byref(p), *dst, None if dwq is None else dwq.data_ptr(),
            None if dwk is None else dwk.data_ptr(), None if ws is None else ws.data_ptr(), need, st))
    return {"dq": rows[0], "dk": rows[1], "dv": rows[2], "dwq": dwq, "dwk": dwk}


def _rows_of(x):
    """(M, K, head_d) of rows [M, K] or of head-major [H, M, d]."""
    if not x.is_cuda:
        raise ValueError("x: device tensor expected")
    if not x.is_contiguous():
        raise ValueError("x: contiguous tensor expected")
    shape = x.shape
    if len(shape) == 2:
        return shape[0], shape[1], 0
    if len(shape) == 3:
        return shape[1], shape[0] * shape[2], shape[2]
    raise ValueError(f"x: [M, K] or [H, M, d] expected, got shape {tuple(shape)}")


def _quantize(x, M, K, head_d, st):
    import torch
    _fits("svgear_mx_quantize", M, K, head_d)
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((M, K // 32), dtype=torch.uint8, device=x.device)
    _check("svgear_mx_quantize", lib().svgear_mx_quantize(
        x.data_ptr(), _code(x.dtype), M, K, head_d, codes.data_ptr(), scales.data_ptr(), st))
    return codes, scales


def _product(pa, psa, M, w_codes, w_scales, bias, dev, st):
    import torch
    N, K, u8 = w_codes.shape[0], w_codes.shape[1] * 2, torch.uint8
    _fits("svgear_mx_product", M, N, K)
    ptrs = (_want("w_codes", w_codes, u8, (N, K // 2), dev), _want("w_scales", w_scales, u8, (N, K // 32), dev),
            _want("bias", bias, torch.float32, (N,), dev))
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _check("svgear_mx_product", lib().svgear_mx_product(pa, psa, *ptrs, M, N, K, y.data_ptr(), st))
    return y


def mx_quantize(x, stream=None):
    """(codes [M, K/2], scales [M, K/32]), uint8, of x [M, K] or of the attention's head-major output
    [H, M, d] (K = H d), through svgear_mx_quantize."""
    M, K, head_d = _rows_of(x)
    with _On(x.device, stream) as st:
        return _quantize(x, M, K, head_d, st)


def mx_dequantize(codes, scales, dtype=None, stream=None):
    """The values [M, K] of codes and scales in `dtype` (default torch.bfloat16), through svgear_mx_dequantize."""
    import torch
    if not codes.is_cuda:
        raise ValueError("codes: device tensor expected")
    if codes.dim() != 2:
        raise ValueError(f"codes: [M, K/2] expected, got shape {tuple(codes.shape)}")
    M, K, dev = codes.shape[0], codes.shape[1] * 2, codes.device
    dtype = dtype or torch.bfloat16
    _fits("svgear_mx_dequantize", M, K)
    pc, ps = _want("codes", codes, torch.uint8, (M, K // 2), dev), _want("scales", scales, torch.uint8, (M, K // 32), dev)
    with _On(dev, stream) as st:
        y = torch.empty((M, K), dtype=dtype, device=dev)
        _check("svgear_mx_dequantize", lib().svgear_mx_dequantize(pc, ps, M, K, y.data_ptr(), _code(dtype), st))
    return y


def mx_product(a_codes, a_scales, w_codes, w_scales, bias=None, stream=None):
    """Y [M, N] bfloat16 = A W^T + bias for MXFP4 A [M, K] and W [N, K], through svgear_mx_product."""
    import torch
    if not a_codes.is_cuda:
        raise ValueError("a_codes: device tensor expected")
    if a_codes.dim() != 2 or w_codes.dim() != 2:
        raise ValueError("a_codes [M, K/2] and w_codes [N, K/2] expected")
    M, K, dev = a_codes.shape[0], w_codes.shape[1] * 2, a_codes.device
    pa = _want("a_codes", a_codes, torch.uint8, (M, K // 2), dev)
    psa = _want("a_scales", a_scales, torch.uint8, (M, K // 32), dev)
    with _On(dev, stream) as st:
        return _product(pa, psa, M, w_codes, w_scales, bias, dev, st)


def mx_linear(x, w_codes, w_scales, bias=None, stream=None):
    """Y [M, N] bfloat16 = quantised x times W^T + bias: mx_quantize, then mx_product."""
    M, K, head_d = _rows_of(x)
    if w_codes.dim() != 2 or K != 2 * w_codes.shape[1]:
        raise ValueError(f"x: {2 * w_codes.shape[-1]} columns expected, got {K}")
    with _On(x.device, stream) as st:
        codes, scales = _quantize(x, M, K, head_d, st)
        return _product(codes.data_ptr(), scales.data_ptr(), M, w_codes, w_scales, bias, x.device, st)

"""ctypes binding for libfab (declared in include/fab.h).

Argument marshalling only: each ``fab_*`` function takes torch CUDA tensors,
checks that they match the layouts the C ABI documents, and passes raw device
pointers, sizes and the current CUDA stream.  Every step of the computation
runs in libfab's kernels; there is no fallback of any kind, and a missing or
unloadable ``libfab.so`` raises.

Tensor shapes (torch, C order; the reverse of ggml's ne order):
    q (B, H, N, DK)  k (B, Hkv, M, DK)  v (B, Hkv, M, DV)
    d, o (B, N, H, DV)  lse (B, H, N) float32  mask (N, M) float16 or None
    packed: float32 of fab_packed_bytes(dims) / 4 elements
    projection rows, read by qk_norm_rope: q (B, N, H, DK)  k (B, N, Hkv, DK)  v (B, N, Hkv, DV),
        heads contiguous, any distance between tokens (views of one fused projection, for example)
    wq, wk (DK,) in q's dtype or None  cos, sin (P, rot / 2) float32  pos (B, N) int32 or None
    paged: projection rows q (T, H, DK)  k (T, Hkv, DK)  v (T, Hkv, DV)
        k_cache (pages, Hkv, page, DK)  v_cache (pages, Hkv, page, DV)
        starts (B + 1,)  lens (B,)  table (B, max_pages), int32;  o (T, H, DV)  lse (H, T) float32
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfab.so")

FAB_OK, FAB_ERR_INVALID, FAB_ERR_UNSUPPORTED, FAB_ERR_WORKSPACE, FAB_ERR_CUDA, FAB_ERR_TIMEOUT = range(6)
FAB_F32, FAB_BF16, FAB_F16 = 0, 1, 2

EXPORTS = ("fab_version", "fab_status_string", "fab_packed_offsets", "fab_packed_bytes",
           "fab_backward_workspace_bytes", "fab_backward_recompute_workspace_bytes", "fab_forward_lse",
           "fab_backward", "fab_backward_preprocess",
           "fab_backward_main", "fab_backward_query_pass", "fab_backward_key_pass", "fab_backward_noalloc",
           "fab_last_device_error", "fab_qk_norm_rope", "fab_qk_norm_rope_backward",
           "fab_qk_norm_rope_backward_workspace_bytes", "fab_paged_append", "fab_paged_attention",
           "fab_paged_attention_workspace_bytes")
NOALLOC_MAX_ROWS = 1048576  # FAB_NOALLOC_MAX_ROWS


class fab_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "H", "Hkv", "N", "M", "DK", "DV")]

    def tuple(self):
        return tuple(getattr(self, n) for n in ("B", "H", "Hkv", "N", "M", "DK", "DV"))


class fab_rope_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "N", "H", "Hkv", "DK", "DV", "rot", "P", "ldq", "ldk", "ldv",
                                              "ldgq", "ldgk", "ldgv")]


class fab_paged_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "H", "Hkv", "DK", "DV", "page", "pages", "max_pages", "rot",
                                              "P", "ldq", "ldk", "ldv")]


class FabError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


_lib = None
_lock = threading.Lock()


def lib():
    """The loaded libfab.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"{LIB_PATH} is missing: build it with attention_backward_tcgen05_gb300.build")
                L = ctypes.CDLL(LIB_PATH)
                vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
                dp = ctypes.POINTER(fab_dims)
                rp, pp = ctypes.POINTER(fab_rope_dims), ctypes.POINTER(fab_paged_dims)
                szp = ctypes.POINTER(ctypes.c_size_t)
                sig = {
                    "fab_version": ([], i32),
                    "fab_status_string": ([i32], ctypes.c_char_p),
                    "fab_packed_offsets": ([dp, szp, szp, szp], i32),
                    "fab_packed_bytes": ([dp], sz),
                    "fab_backward_workspace_bytes": ([dp, i32], sz),
                    "fab_backward_recompute_workspace_bytes": ([dp, i32], sz),
                    "fab_forward_lse": ([vp, vp, vp, vp, i32, f32, i32, dp, vp, vp, vp], i32),
                    "fab_backward": ([vp, vp, vp, vp, vp, vp, vp, i32, f32, i32, dp, vp, sz, vp, vp], i32),
                    "fab_backward_preprocess": ([vp, vp, i32, dp, vp, sz, vp, vp], i32),
                    "fab_backward_main": ([vp, vp, vp, vp, vp, vp, i32, f32, i32, dp, vp, sz, vp, vp], i32),
                    "fab_backward_query_pass": ([vp, vp, vp, vp, vp, vp, vp, i32, f32, i32, dp, vp, sz, vp, vp], i32),
                    "fab_backward_key_pass": ([vp, vp, vp, vp, vp, vp, i32, f32, i32, dp, vp, sz, vp, vp], i32),
                    "fab_backward_noalloc": ([vp, vp, vp, vp, vp, vp, vp, i32, f32, i32, dp, vp, vp], i32),
                    "fab_last_device_error": ([vp], i32),
                    "fab_qk_norm_rope": ([vp] * 8 + [f32, i32, i32, rp, vp, vp, vp, vp], i32),
                    "fab_qk_norm_rope_backward_workspace_bytes": ([rp], sz),
                    "fab_qk_norm_rope_backward": ([vp] * 10 + [f32, i32, i32, rp, vp, sz] + [vp] * 6, i32),
                    "fab_paged_append": ([vp] * 7 + [f32, i32, vp, vp, vp, i32, pp, vp, vp, vp, vp], i32),
                    "fab_paged_attention_workspace_bytes": ([pp, i32], sz),
                    "fab_paged_attention": ([vp] * 6 + [i32, f32, i32, pp, vp, sz, vp, vp, vp], i32),
                }
                for name, (args, res) in sig.items():
                    f = getattr(L, name)
                    f.argtypes = args
                    f.restype = res
                _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().fab_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != FAB_OK:
        raise FabError(status, where)


def make_dims(B, H, Hkv, N, M, DK, DV) -> fab_dims:
    return fab_dims(int(B), int(H), int(Hkv), int(N), int(M), int(DK), int(DV))


def dims_of(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> fab_dims:
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D: (B,H,N,DK), (B,Hkv,M,DK), (B,Hkv,M,DV)")
    B, H, N, DK = q.shape
    Bk, Hkv, M, DKk = k.shape
    Bv, Hv, Mv, DV = v.shape
    if (Bk, DKk) != (B, DK) or (Bv, Hv, Mv) != (B, Hkv, M):
        raise ValueError("inconsistent q/k/v shapes")
    return make_dims(B, H, Hkv, N, M, DK, DV)


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return FAB_F32
    if t.dtype == torch.bfloat16:
        return FAB_BF16
    if t.dtype == torch.float16:
        return FAB_F16
    raise ValueError(f"unsupported dtype {t.dtype}: float32, bfloat16 or float16")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev(t: torch.Tensor, name: str, dtype=None, shape=None) -> ctypes.c_void_p:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _mask(mask, dims: fab_dims):
    if mask is None:
        return None
    return _dev(mask, "mask", torch.float16, (dims.N, dims.M))


# ------------------------------------------------------------------ C ABI, one to one


def fab_version() -> int:
    return lib().fab_version()


def fab_packed_offsets(dims: fab_dims):
    a, b, c = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().fab_packed_offsets(ctypes.byref(dims), ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
           "fab_packed_offsets")
    return a.value, b.value, c.value


def fab_packed_bytes(dims: fab_dims) -> int:
    return lib().fab_packed_bytes(ctypes.byref(dims))


def fab_backward_workspace_bytes(dims: fab_dims, dtype: int) -> int:
    return lib().fab_backward_workspace_bytes(ctypes.byref(dims), int(dtype))


def fab_backward_recompute_workspace_bytes(dims: fab_dims, dtype: int) -> int:
    return lib().fab_backward_recompute_workspace_bytes(ctypes.byref(dims), int(dtype))


def fab_forward_lse(q, k, v, mask, causal, scale, o, lse, stream=None):
    dims = dims_of(q, k, v)
    t = dtype_code(q)
    args = (_dev(q, "q"), _dev(k, "k", q.dtype), _dev(v, "v", q.dtype), _mask(mask, dims), int(bool(causal)),
            float(scale), t, ctypes.byref(dims),
            _dev(o, "o", q.dtype, (dims.B, dims.N, dims.H, dims.DV)),
            _dev(lse, "lse", torch.float32, (dims.B, dims.H, dims.N)), _stream(stream))
    _check(lib().fab_forward_lse(*args), "fab_forward_lse")


def fab_backward(q, k, v, d, o, lse, mask, causal, scale, workspace, packed_out, stream=None):
    """o and lse may both be None: the library then recomputes them into the
    workspace (sized by fab_backward_recompute_workspace_bytes)."""
    dims = dims_of(q, k, v)
    t = dtype_code(q)
    oshape = (dims.B, dims.N, dims.H, dims.DV)
    args = (_dev(q, "q"), _dev(k, "k", q.dtype), _dev(v, "v", q.dtype), _dev(d, "d", q.dtype, oshape),
            None if o is None else _dev(o, "o", q.dtype, oshape),
            None if lse is None else _dev(lse, "lse", torch.float32, (dims.B, dims.H, dims.N)),
            _mask(mask, dims), int(bool(causal)), float(scale), t, ctypes.byref(dims),
            _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
            _dev(packed_out, "packed_out", torch.float32, (fab_packed_bytes(dims) // 4,)), _stream(stream))
    _check(lib().fab_backward(*args), "fab_backward")


def fab_backward_preprocess(d, o, dims: fab_dims, workspace, packed_out, stream=None):
    oshape = (dims.B, dims.N, dims.H, dims.DV)
    t = dtype_code(d)
    args = (_dev(d, "d", None, oshape), _dev(o, "o", d.dtype, oshape), t, ctypes.byref(dims),
            _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
            _dev(packed_out, "packed_out", torch.float32, (fab_packed_bytes(dims) // 4,)), _stream(stream))
    _check(lib().fab_backward_preprocess(*args), "fab_backward_preprocess")


def fab_backward_main(q, k, v, d, lse, mask, causal, scale, workspace, packed_out, stream=None):
    dims = dims_of(q, k, v)
    t = dtype_code(q)
    args = (_dev(q, "q"), _dev(k, "k", q.dtype), _dev(v, "v", q.dtype),
            _dev(d, "d", q.dtype, (dims.B, dims.N, dims.H, dims.DV)),
            _dev(lse, "lse", torch.float32, (dims.B, dims.H, dims.N)), _mask(mask, dims), int(bool(causal)),
            float(scale), t, ctypes.byref(dims), _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size(),
            _dev(packed_out, "packed_out", torch.float32, (fab_packed_bytes(dims) // 4,)), _stream(stream))
    _check(lib().fab_backward_main(*args), "fab_backward_main")


def fab_backward_query_pass(q, k, v, d, o, lse, mask, causal, scale, workspace, packed_out, stream=None):
    """Tensor-core query pass: D_i into the workspace, the dQ slice and the padding."""
    dims = dims_of(q, k, v)
    t = dtype_code(q)
    oshape = (dims.B, dims.N, dims.H, dims.DV)
    args = (_dev(q, "q"), _dev(k, "k", q.dtype), _dev(v, "v", q.dtype), _dev(d, "d", q.dtype, oshape),
            _dev(o, "o", q.dtype, oshape), _dev(lse, "lse", torch.float32, (dims.B, dims.H, dims.N)),
            _mask(mask, dims), int(bool(causal)), float(scale), t, ctypes.byref(dims),
            _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
            _dev(packed_out, "packed_out", torch.float32, (fab_packed_bytes(dims) // 4,)), _stream(stream))
    _check(lib().fab_backward_query_pass(*args), "fab_backward_query_pass")


def fab_backward_key_pass(q, k, v, d, lse, mask, causal, scale, workspace, packed_out, stream=None):
    """Tensor-core key/value pass: the dK and dV slices (D_i read from the workspace)."""
    dims = dims_of(q, k, v)
    t = dtype_code(q)
    args = (_dev(q, "q"), _dev(k, "k", q.dtype), _dev(v, "v", q.dtype),
            _dev(d, "d", q.dtype, (dims.B, dims.N, dims.H, dims.DV)),
            _dev(lse, "lse", torch.float32, (dims.B, dims.H, dims.N)), _mask(mask, dims), int(bool(causal)),
            float(scale), t, ctypes.byref(dims), _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size(),
            _dev(packed_out, "packed_out", torch.float32, (fab_packed_bytes(dims) // 4,)), _stream(stream))
    _check(lib().fab_backward_key_pass(*args), "fab_backward_key_pass")


def fab_backward_noalloc(q, k, v, d, o, lse, mask, causal, scale, packed_out, stream=None):
    """fab_backward without a workspace: for callers that cannot allocate
    device memory.  The scratch is a fixed array inside libfab (B*H*N up to
    NOALLOC_MAX_ROWS); calls that may overlap on the GPU must be ordered."""
    dims = dims_of(q, k, v)
    t = dtype_code(q)
    oshape = (dims.B, dims.N, dims.H, dims.DV)
    args = (_dev(q, "q"), _dev(k, "k", q.dtype), _dev(v, "v", q.dtype), _dev(d, "d", q.dtype, oshape),
            _dev(o, "o", q.dtype, oshape), _dev(lse, "lse", torch.float32, (dims.B, dims.H, dims.N)),
            _mask(mask, dims), int(bool(causal)), float(scale), t, ctypes.byref(dims),
            _dev(packed_out, "packed_out", torch.float32, (fab_packed_bytes(dims) // 4,)), _stream(stream))
    _check(lib().fab_backward_noalloc(*args), "fab_backward_noalloc")


def fab_last_device_error(stream=None) -> int:
    return lib().fab_last_device_error(_stream(stream))


# ------------------------------------------------------------------ norms + rotation, paged cache


# A small call's time is its host's: these checks ask each tensor for each
# property once.


def _here(*tensors):
    """All the given tensors (None: skipped) are on the current device, which
    is where libfab launches; returns that device's index."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {tensors[0].device} and {t.device}")
    if dev < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if dev != torch.cuda.current_device():
        raise ValueError(f"tensors on cuda:{dev}, but the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _ptr(t, name, dtype, shape):
    """Address of a contiguous tensor of that dtype and shape (None: null)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, {dtype}, of shape {tuple(shape)}; "
                         f"got {t.dtype} {tuple(t.shape)} strides {t.stride()}")
    return t.data_ptr()


def _ld(t, name, dtype, shape):
    """Elements between the rows of consecutive tokens of t, of shape
    (..., tokens, heads, width): heads contiguous inside a row, rows evenly
    spaced over all tokens."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    st = t.stride()
    heads, width = shape[-2], shape[-1]
    if (st[-1] != 1 and width > 1) or (st[-2] != width and heads > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous, got strides {st}")
    n = shape[-3]
    if len(shape) == 4 and shape[0] > 1:
        if n == 1:
            return st[0]
        if st[0] != n * st[1]:
            raise ValueError(f"{name}: the rows of all tokens must be evenly spaced, got strides {st}")
    return st[-3] if n > 1 else heads * width


def _tables(cos, sin, wq, wk, DK, dtype):
    """(rot, P, addresses of wq, wk, cos, sin); without cos and sin no rotation."""
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    w = _ptr(wq, "wq", dtype, (DK,)), _ptr(wk, "wk", dtype, (DK,))
    if cos is None:
        return 0, 0, (*w, None, None)
    shape = cos.shape
    if len(shape) != 2:
        raise ValueError("cos, sin must be 2-D: (P,rot/2)")
    f32 = torch.float32
    return 2 * shape[1], shape[0], (*w, _ptr(cos, "cos", f32, shape), _ptr(sin, "sin", f32, shape))


def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, dev):
    """As _stream, without building a Stream object for the current one (3 us
    a call on the host, more than a small launch takes)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def fab_qk_norm_rope(q, k, v, wq, wk, cos, sin, pos, eps, interleaved, q_out, k_out, v_out, stream=None):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k must be 4-D: (B,N,H,DK), (B,N,Hkv,DK)")
    qs = q.shape
    B, N, H, DK = qs
    Hkv = k.shape[2]
    dt = q.dtype
    code = dtype_code(q)
    dev = _here(q, k, v, wq, wk, cos, sin, pos, q_out, k_out, v_out)
    rot, P, tables = _tables(cos, sin, wq, wk, DK, dt)
    DV, ldv, vp, vo = DK, 0, None, None
    if v is not None:
        DV = v.shape[-1]
        ldv, vp = _ld(v, "v", dt, (B, N, Hkv, DV)), v.data_ptr()
    if v_out is not None:
        vo = _ptr(v_out, "v_out", dt, (B, Hkv, N, DV))
    dims = fab_rope_dims(B, N, H, Hkv, DK, DV, rot, P, _ld(q, "q", dt, qs), _ld(k, "k", dt, (B, N, Hkv, DK)), ldv)
    _check(lib().fab_qk_norm_rope(
        q.data_ptr(), k.data_ptr(), vp, *tables, _ptr(pos, "pos", torch.int32, (B, N)), eps, 1 if interleaved else 0,
        code, ctypes.byref(dims), _ptr(q_out, "q_out", dt, (B, H, N, DK)), _ptr(k_out, "k_out", dt, (B, Hkv, N, DK)),
        vo, _raw_stream(stream, dev)), "fab_qk_norm_rope")


def fab_qk_norm_rope_backward_workspace_bytes(dims: fab_rope_dims) -> int:
    return lib().fab_qk_norm_rope_backward_workspace_bytes(ctypes.byref(dims))


def _rope_backward_dims(dq, dk, dv, q, k, wq, wk, rot, P, gq, gk, gv):
    B, H, N, DK = dq.shape
    Hkv, DV = dk.shape[1], DK if dv is None else dv.shape[-1]
    dt = gq.dtype
    qs, ks = (B, N, H, DK), (B, N, Hkv, DK)
    return fab_rope_dims(B, N, H, Hkv, DK, DV, rot, P, 0 if wq is None else _ld(q, "q", dt, qs),
                         0 if wk is None else _ld(k, "k", dt, ks), 0, _ld(gq, "gq", dt, qs), _ld(gk, "gk", dt, ks),
                         0 if gv is None else _ld(gv, "gv", dt, (B, N, Hkv, DV)))


def fab_qk_norm_rope_backward(dq, dk, dv, q, k, wq, wk, cos, sin, pos, eps, interleaved, workspace, gq, gk, gv, gwq,
                              gwk, stream=None):
    """q and k are read only where wq and wk are given (None otherwise is fine)."""
    if dq.dim() != 4 or dk.dim() != 4:
        raise ValueError("dq, dk must be 4-D: (B,H,N,DK), (B,Hkv,N,DK)")
    B, H, N, DK = dq.shape
    dev = _here(dq, dk, dv, q, k, wq, wk, cos, sin, pos, workspace, gq, gk, gv, gwq, gwk)
    rot, P, tables = _tables(cos, sin, wq, wk, DK, gq.dtype)
    dims = _rope_backward_dims(dq, dk, dv, q, k, wq, wk, rot, P, gq, gk, gv)
    f32 = torch.float32
    _check(lib().fab_qk_norm_rope_backward(
        _ptr(dq, "dq", f32, dq.shape), _ptr(dk, "dk", f32, (B, dims.Hkv, N, DK)),
        _ptr(dv, "dv", f32, (B, dims.Hkv, N, dims.DV)), None if wq is None else q.data_ptr(),
        None if wk is None else k.data_ptr(), *tables,
        _ptr(pos, "pos", torch.int32, (B, N)), eps, 1 if interleaved else 0, dtype_code(gq),
        ctypes.byref(dims), _addr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), gq.data_ptr(), gk.data_ptr(),
        _addr(gv), _ptr(gwq, "gwq", f32, (DK,)), _ptr(gwk, "gwk", f32, (DK,)), _raw_stream(stream, dev)),
        "fab_qk_norm_rope_backward")


def _paged_dims(H, T, k_cache, v_cache, starts, lens, table):
    """dims of a paged call, its cache and its int32 arrays checked."""
    if k_cache.dim() != 4 or v_cache.dim() != 4 or table.dim() != 2:
        raise ValueError("k_cache, v_cache must be 4-D (pages,Hkv,page,width), table 2-D (B,max_pages)")
    pages, Hkv, page, DK = k_cache.shape
    DV = v_cache.shape[3]
    B, max_pages = table.shape
    _ptr(k_cache, "k_cache", k_cache.dtype, k_cache.shape)
    _ptr(v_cache, "v_cache", k_cache.dtype, (pages, Hkv, page, DV))
    i32 = torch.int32
    _ptr(starts, "starts", i32, (B + 1,))
    _ptr(lens, "lens", i32, (B,))
    _ptr(table, "table", i32, (B, max_pages))
    return fab_paged_dims(B, T, H, Hkv, DK, DV, page, pages, max_pages)


def fab_paged_append(q, k, v, wq, wk, cos, sin, eps, interleaved, starts, lens, table, q_out, k_cache, v_cache,
                     stream=None):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be 3-D: (T,H,DK), (T,Hkv,DK), (T,Hkv,DV)")
    T, H, DK = q.shape
    dt = q.dtype
    dev = _here(q, k, v, wq, wk, cos, sin, starts, lens, table, q_out, k_cache, v_cache)
    dims = _paged_dims(H, T, k_cache, v_cache, starts, lens, table)
    if k_cache.dtype != dt:
        raise ValueError(f"k_cache must be {dt}, got {k_cache.dtype}")
    dims.rot, dims.P, tables = _tables(cos, sin, wq, wk, DK, dt)
    dims.ldq = _ld(q, "q", dt, (T, H, dims.DK))
    dims.ldk = _ld(k, "k", dt, (T, dims.Hkv, DK))
    dims.ldv = _ld(v, "v", dt, (T, dims.Hkv, dims.DV))
    _check(lib().fab_paged_append(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), *tables, eps, 1 if interleaved else 0, starts.data_ptr(),
        lens.data_ptr(), table.data_ptr(), dtype_code(q), ctypes.byref(dims), _ptr(q_out, "q_out", dt, (T, H, DK)),
        k_cache.data_ptr(), v_cache.data_ptr(), _raw_stream(stream, dev)), "fab_paged_append")


def fab_paged_attention_workspace_bytes(dims: fab_paged_dims, dtype: int) -> int:
    return lib().fab_paged_attention_workspace_bytes(ctypes.byref(dims), int(dtype))


def fab_paged_attention(q, k_cache, v_cache, starts, lens, table, causal, scale, workspace, o, lse, stream=None):
    """lse may be None."""
    if q.dim() != 3:
        raise ValueError("q must be 3-D: (T,H,DK)")
    T, H, DK = q.shape
    dt = q.dtype
    dev = _here(q, k_cache, v_cache, starts, lens, table, workspace, o, lse)
    dims = _paged_dims(H, T, k_cache, v_cache, starts, lens, table)
    if k_cache.dtype != dt:
        raise ValueError(f"k_cache must be {dt}, got {k_cache.dtype}")
    _check(lib().fab_paged_attention(
        _ptr(q, "q", dt, (T, H, dims.DK)), k_cache.data_ptr(), v_cache.data_ptr(), starts.data_ptr(),
        lens.data_ptr(), table.data_ptr(), int(bool(causal)), float(scale), dtype_code(q), ctypes.byref(dims),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _ptr(o, "o", dt, (T, H, dims.DV)),
        _ptr(lse, "lse", torch.float32, (H, T)), _raw_stream(stream, dev)), "fab_paged_attention")


# ------------------------------------------------------------------ conveniences (torch allocates, libfab computes)


def _on(stream):
    """A context whose allocations belong to `stream` (None: the current one),
    so that torch does not hand their memory to other work too early."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


@functools.lru_cache(maxsize=256)
def _rope_workspace(B, N, H, Hkv, DK):
    return max(fab_qk_norm_rope_backward_workspace_bytes(fab_rope_dims(B, N, H, Hkv, DK, DK)), 16)


@functools.lru_cache(maxsize=256)
def _paged_workspace(dtype, *dims):
    return max(fab_paged_attention_workspace_bytes(fab_paged_dims(*dims), dtype), 16)


def qk_norm_rope(q, k, v, wq=None, wk=None, cos=None, sin=None, pos=None, eps=1e-6, interleaved=False, stream=None):
    """Projection rows q (B,N,H,DK), k (B,N,Hkv,DK), v (B,N,Hkv,DV) or None to
    what forward() takes: q (B,H,N,DK), k (B,Hkv,N,DK) normalised per head
    (where weights are given) and rotated (where tables are), v (B,Hkv,N,DV)."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k must be 4-D: (B,N,H,DK), (B,N,Hkv,DK)")
    B, N, H, DK = q.shape
    with _on(stream):
        dt, dev = q.dtype, q.device
        qo = torch.empty((B, H, N, DK), dtype=dt, device=dev)
        ko = torch.empty((B, k.shape[2], N, DK), dtype=dt, device=dev)
        vo = None if v is None else torch.empty((B, v.shape[2], N, v.shape[3]), dtype=dt, device=dev)
        fab_qk_norm_rope(q, k, v, wq, wk, cos, sin, pos, eps, interleaved, qo, ko, vo, stream)
    return qo, ko, vo


def qk_norm_rope_backward(dq, dk, dv, q, k, wq=None, wk=None, cos=None, sin=None, pos=None, eps=1e-6,
                          interleaved=False, dtype=None, stream=None):
    """The gradients of qk_norm_rope's q, k, v, wq, wk for those of its results
    (unpack()'s float32 slices): (gq (B,N,H,DK), gk (B,N,Hkv,DK), gv (B,N,Hkv,DV)
    or None, gwq, gwk float32 (DK,) or None).  gq, gk and gv are in `dtype`
    (None: q's) and are views of one row of H*DK + Hkv*DK + Hkv*DV values a
    token: gq._base is the gradient of a fused projection."""
    if dq.dim() != 4 or dk.dim() != 4:
        raise ValueError("dq, dk must be 4-D: (B,H,N,DK), (B,Hkv,N,DK)")
    B, H, N, DK = dq.shape
    Hkv = dk.shape[1]
    dtype = q.dtype if dtype is None else dtype
    nq, nk, nv = H * DK, Hkv * DK, 0 if dv is None else dv.shape[1] * dv.shape[3]
    with _on(stream):
        g = torch.empty((B, N, nq + nk + nv), dtype=dtype, device=dq.device)
        gq = g.as_strided((B, N, H, DK), (N * g.shape[2], g.shape[2], DK, 1))
        gk = g.as_strided((B, N, Hkv, DK), (N * g.shape[2], g.shape[2], DK, 1), nq)
        gv = None
        if dv is not None:
            gv = g.as_strided((B, N, dv.shape[1], dv.shape[3]), (N * g.shape[2], g.shape[2], dv.shape[3], 1), nq + nk)
        gwq = None if wq is None else torch.empty((DK,), dtype=torch.float32, device=dq.device)
        gwk = None if wk is None else torch.empty((DK,), dtype=torch.float32, device=dq.device)
        ws = None
        if wq is not None or wk is not None:
            ws = torch.empty(_rope_workspace(B, N, H, Hkv, DK), dtype=torch.uint8, device=dq.device)
        fab_qk_norm_rope_backward(dq, dk, dv, q, k, wq, wk, cos, sin, pos, eps, interleaved, ws, gq, gk, gv, gwq, gwk,
                                  stream)
    return gq, gk, gv, gwq, gwk


def paged_append(q, k, v, wq, wk, cos, sin, starts, lens, table, k_cache, v_cache, eps=1e-6, interleaved=False,
                 stream=None):
    """Puts the new tokens' keys and values into the caches and returns their
    queries (T,H,DK), normalised and rotated as qk_norm_rope does; rows of
    padding tokens are left as allocated."""
    with _on(stream):
        qo = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        fab_paged_append(q, k, v, wq, wk, cos, sin, eps, interleaved, starts, lens, table, qo, k_cache, v_cache, stream)
    return qo


def alloc_paged(q, k_cache, v_cache, table):
    """A workspace (uint8 tensor) for fab_paged_attention calls of these sizes."""
    pages, Hkv, page, DK = k_cache.shape
    B, max_pages = table.shape
    wsb = _paged_workspace(dtype_code(q), B, q.shape[0], q.shape[1], Hkv, DK, v_cache.shape[3], page, pages, max_pages)
    return torch.empty(wsb, dtype=torch.uint8, device=q.device)


def paged_attention(q, k_cache, v_cache, starts, lens, table, causal=True, scale=None, stream=None):
    """Returns (o (T,H,DV) in q's dtype, lse (H,T) float32); rows of padding
    tokens are left as allocated."""
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    with _on(stream):
        T, H, dev = q.shape[0], q.shape[1], q.device
        o = torch.empty((T, H, v_cache.shape[-1]), dtype=q.dtype, device=dev)
        lse = torch.empty((H, T), dtype=torch.float32, device=dev)
        ws = alloc_paged(q, k_cache, v_cache, table)
        fab_paged_attention(q, k_cache, v_cache, starts, lens, table, causal, scale, ws, o, lse, stream)
    return o, lse




def forward(q, k, v, mask=None, causal=False, scale=None, stream=None):
    """Returns (o (B,N,H,DV) in q's dtype, lse (B,H,N) float32)."""
    dims = dims_of(q, k, v)
    scale = dims.DK ** -0.5 if scale is None else scale
    o = torch.empty((dims.B, dims.N, dims.H, dims.DV), dtype=q.dtype, device=q.device)
    lse = torch.empty((dims.B, dims.H, dims.N), dtype=torch.float32, device=q.device)
    fab_forward_lse(q, k, v, mask, causal, scale, o, lse, stream)
    return o, lse


def alloc_backward(dims: fab_dims, dtype: int, device, recompute: bool = False):
    """(workspace uint8 tensor, packed float32 tensor) sized for fab_backward
    (recompute: for a call without o and lse)."""
    wsb = fab_backward_recompute_workspace_bytes(dims, dtype) if recompute else fab_backward_workspace_bytes(dims, dtype)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=device)
    packed = torch.empty(fab_packed_bytes(dims) // 4, dtype=torch.float32, device=device)
    return ws, packed


def backward(q, k, v, d, o=None, lse=None, mask=None, causal=False, scale=None, stream=None):
    """Returns the packed f32 [dQ | dK | dV] buffer (o, lse None: recomputed)."""
    dims = dims_of(q, k, v)
    scale = dims.DK ** -0.5 if scale is None else scale
    ws, packed = alloc_backward(dims, dtype_code(q), q.device, recompute=o is None and lse is None)
    fab_backward(q, k, v, d, o, lse, mask, causal, scale, ws, packed, stream)
    return packed


def unpack(packed: torch.Tensor, dims: fab_dims):
    """Views (dq (B,H,N,DK), dk (B,Hkv,M,DK), dv (B,Hkv,M,DV)) into a packed buffer."""
    off_k, off_v, end = fab_packed_offsets(dims)
    B, H, Hkv, N, M, DK, DV = dims.tuple()
    nq, nk, nv = B * H * N * DK, B * Hkv * M * DK, B * Hkv * M * DV
    dq = packed[:nq].view(B, H, N, DK)
    dk = packed[off_k // 4:off_k // 4 + nk].view(B, Hkv, M, DK)
    dv = packed[off_v // 4:off_v // 4 + nv].view(B, Hkv, M, DV)
    return dq, dk, dv

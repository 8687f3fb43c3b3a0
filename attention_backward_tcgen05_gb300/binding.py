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


# A small call's time is its host's.  What a call checks and hands over depends
# on its tensors' layouts alone, so it is worked out once for each set of them
# (`_layouts`, the functions under `functools.lru_cache`): a training step's
# or a decoding loop's calls find it by one look-up.


def _layouts(*tensors):
    """(shape, strides, dtype, device) of each tensor; None of None."""
    return tuple([None if t is None else (t.shape, t.stride(), t.dtype, t.get_device()) for t in tensors])


def _one_device(layouts):
    """The device index that all the given layouts (None: skipped) share."""
    devs = {x[3] for x in layouts if x is not None}
    if min(devs) < 0:
        raise ValueError("the tensors must be CUDA tensors")
    if len(devs) > 1:
        raise ValueError(f"tensors on {sorted(f'cuda:{d}' for d in devs)}")
    return devs.pop()


def _current(dev):
    """libfab launches on the current device: it has to be the tensors'."""
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on cuda:{dev}, but the current device is cuda:{torch.cuda.current_device()}")


def _whole(x, name, dtype, shape):
    """Checks that a layout (None: skipped) is contiguous, of that dtype and shape."""
    if x is None:
        return
    shape = tuple(shape)
    ok = x[2] is dtype and x[0] == shape
    if ok and 0 not in shape:
        step = 1
        for n, st in zip(reversed(shape), reversed(x[1])):
            ok = ok and (n == 1 or st == step)
            step *= n
    if not ok:
        raise ValueError(f"{name} must be contiguous, {dtype}, of shape {shape}; "
                         f"got {x[2]} {tuple(x[0])} strides {x[1]}")


def _outputs(dev, *checks):
    """Each (tensor or None, name, dtype, shape) is whole and on device dev."""
    for t, name, dtype, shape in checks:
        if t is not None:
            _whole((t.shape, t.stride(), t.dtype, dev), name, dtype, shape)
            if t.get_device() != dev:
                raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{dev}")


def _ld(x, name, dtype, shape):
    """Elements between the rows of consecutive tokens of a layout of shape
    (..., tokens, heads, width): heads contiguous inside a row, rows evenly
    spaced over all tokens."""
    if x[2] is not dtype or x[0] != tuple(shape):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {x[2]} {tuple(x[0])}")
    st = x[1]
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
    """(rot, P) of the tables' layouts, checked with the weights'; without cos and sin no rotation."""
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    _whole(wq, "wq", dtype, (DK,))
    _whole(wk, "wk", dtype, (DK,))
    if cos is None:
        return 0, 0
    shape = cos[0]
    if len(shape) != 2:
        raise ValueError("cos, sin must be 2-D: (P,rot/2)")
    _whole(cos, "cos", torch.float32, shape)
    _whole(sin, "sin", torch.float32, shape)
    return 2 * shape[1], shape[0]


def _code(dtype):
    try:
        return {torch.float32: FAB_F32, torch.bfloat16: FAB_BF16, torch.float16: FAB_F16}[dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {dtype}: float32, bfloat16 or float16") from None


def _bytes(workspace, dev):
    """Bytes of a workspace (None: 0), which has to be on device dev."""
    if workspace is None:
        return 0
    if workspace.get_device() != dev:
        raise ValueError(f"the workspace is on {workspace.device}, the other tensors on cuda:{dev}")
    if not workspace.is_contiguous():  # (its elements' bytes are not then those from its address on)
        raise ValueError(f"the workspace must be contiguous, got strides {workspace.stride()}")
    return workspace.numel() * workspace.element_size()


def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, dev):
    """As _stream, without building a Stream object for the current one (3 us
    a call on the host, more than a small launch takes)."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


@functools.lru_cache(maxsize=1024)
def _rope_plan(layouts):
    """(dims, their reference, dtype code, device) of a fab_qk_norm_rope call on
    q, k, v, wq, wk, cos, sin, pos."""
    q, k, v, wq, wk, cos, sin, pos = layouts
    if len(q[0]) != 4 or len(k[0]) != 4:
        raise ValueError("q, k must be 4-D: (B,N,H,DK), (B,N,Hkv,DK)")
    B, N, H, DK = q[0]
    Hkv = k[0][2]
    dt = q[2]
    code = _code(dt)
    dev = _one_device(layouts)
    rot, P = _tables(cos, sin, wq, wk, DK, dt)
    DV, ldv = DK, 0
    if v is not None:
        DV = v[0][-1]
        ldv = _ld(v, "v", dt, (B, N, Hkv, DV))
    _whole(pos, "pos", torch.int32, (B, N))
    dims = fab_rope_dims(B, N, H, Hkv, DK, DV, rot, P, _ld(q, "q", dt, q[0]), _ld(k, "k", dt, (B, N, Hkv, DK)), ldv)
    return dims, ctypes.byref(dims), code, dev


def _rope_call(plan, q, k, v, wq, wk, cos, sin, pos, eps, interleaved, q_out, k_out, v_out, stream):
    dev = plan[3]
    _current(dev)
    _check(lib().fab_qk_norm_rope(
        q.data_ptr(), k.data_ptr(), _addr(v), _addr(wq), _addr(wk), _addr(cos), _addr(sin), _addr(pos), eps,
        1 if interleaved else 0, plan[2], plan[1], q_out.data_ptr(), k_out.data_ptr(), _addr(v_out),
        _raw_stream(stream, dev)), "fab_qk_norm_rope")


def fab_qk_norm_rope(q, k, v, wq, wk, cos, sin, pos, eps, interleaved, q_out, k_out, v_out, stream=None):
    plan = _rope_plan(_layouts(q, k, v, wq, wk, cos, sin, pos))
    d, dt = plan[0], q.dtype
    _outputs(plan[3], (q_out, "q_out", dt, (d.B, d.H, d.N, d.DK)), (k_out, "k_out", dt, (d.B, d.Hkv, d.N, d.DK)),
             (v_out, "v_out", dt, (d.B, d.Hkv, d.N, d.DV)))
    _rope_call(plan, q, k, v, wq, wk, cos, sin, pos, eps, interleaved, q_out, k_out, v_out, stream)


def fab_qk_norm_rope_backward_workspace_bytes(dims: fab_rope_dims) -> int:
    return lib().fab_qk_norm_rope_backward_workspace_bytes(ctypes.byref(dims))


@functools.lru_cache(maxsize=1024)
def _rope_backward_plan(layouts, dt, out):
    """(dims, their reference, dtype code, device, workspace bytes) of a
    fab_qk_norm_rope_backward call on dq, dk, dv, q, k, wq, wk, cos, sin, pos.
    out: the layouts of gq, gk, gv, or None: one row holds all three."""
    dq, dk, dv, q, k, wq, wk, cos, sin, pos = layouts
    if len(dq[0]) != 4 or len(dk[0]) != 4:
        raise ValueError("dq, dk must be 4-D: (B,H,N,DK), (B,Hkv,N,DK)")
    B, H, N, DK = dq[0]
    Hkv, DV = dk[0][1], DK if dv is None else dv[0][-1]
    dev = _one_device(layouts if out is None else layouts + out)
    rot, P = _tables(cos, sin, wq, wk, DK, dt)
    f32 = torch.float32
    _whole(dq, "dq", f32, dq[0])
    _whole(dk, "dk", f32, (B, Hkv, N, DK))
    _whole(dv, "dv", f32, (B, Hkv, N, DV))
    _whole(pos, "pos", torch.int32, (B, N))
    if (wq is not None and q is None) or (wk is not None and k is None):
        raise ValueError("q and k are needed where wq and wk are given")
    qs, ks, vs = (B, N, H, DK), (B, N, Hkv, DK), (B, N, Hkv, DV)
    ldq, ldk = 0 if wq is None else _ld(q, "q", dt, qs), 0 if wk is None else _ld(k, "k", dt, ks)
    if out is None:
        ldg = [H * DK + Hkv * DK + (0 if dv is None else Hkv * DV)] * 3
    else:
        ldg = [0 if x is None else _ld(x, *to) for x, to in zip(out, (("gq", dt, qs), ("gk", dt, ks), ("gv", dt, vs)))]
    dims = fab_rope_dims(B, N, H, Hkv, DK, DV, rot, P, ldq, ldk, 0, *ldg)
    return dims, ctypes.byref(dims), _code(dt), dev, fab_qk_norm_rope_backward_workspace_bytes(dims)


def _rope_backward_call(plan, dq, dk, dv, q, k, wq, wk, cos, sin, pos, eps, interleaved, ws, wsb, gq, gk, gv, gwq, gwk,
                        stream):
    dev = plan[3]
    _current(dev)
    _check(lib().fab_qk_norm_rope_backward(
        dq.data_ptr(), dk.data_ptr(), _addr(dv), None if wq is None else q.data_ptr(),
        None if wk is None else k.data_ptr(), _addr(wq), _addr(wk), _addr(cos), _addr(sin), _addr(pos), eps,
        1 if interleaved else 0, plan[2], plan[1], _addr(ws), wsb, gq.data_ptr(), gk.data_ptr(), _addr(gv), _addr(gwq),
        _addr(gwk), _raw_stream(stream, dev)), "fab_qk_norm_rope_backward")


def fab_qk_norm_rope_backward(dq, dk, dv, q, k, wq, wk, cos, sin, pos, eps, interleaved, workspace, gq, gk, gv, gwq,
                              gwk, stream=None):
    """q and k are read only where wq and wk are given (None otherwise is fine)."""
    plan = _rope_backward_plan(_layouts(dq, dk, dv, q, k, wq, wk, cos, sin, pos), gq.dtype, _layouts(gq, gk, gv))
    f32, DK = torch.float32, plan[0].DK
    _outputs(plan[3], (gwq, "gwq", f32, (DK,)), (gwk, "gwk", f32, (DK,)))
    _rope_backward_call(plan, dq, dk, dv, q, k, wq, wk, cos, sin, pos, eps, interleaved, workspace,
                        _bytes(workspace, plan[3]), gq, gk, gv, gwq, gwk, stream)


def _paged_dims(H, T, dt, k_cache, v_cache, starts, lens, table):
    """dims of a paged call, the layouts of its cache and its int32 arrays checked."""
    if len(k_cache[0]) != 4 or len(v_cache[0]) != 4 or len(table[0]) != 2:
        raise ValueError("k_cache, v_cache must be 4-D (pages,Hkv,page,width), table 2-D (B,max_pages)")
    pages, Hkv, page, DK = k_cache[0]
    DV = v_cache[0][3]
    B, max_pages = table[0]
    _whole(k_cache, "k_cache", dt, k_cache[0])
    _whole(v_cache, "v_cache", dt, (pages, Hkv, page, DV))
    i32 = torch.int32
    _whole(starts, "starts", i32, (B + 1,))
    _whole(lens, "lens", i32, (B,))
    _whole(table, "table", i32, (B, max_pages))
    return fab_paged_dims(B, T, H, Hkv, DK, DV, page, pages, max_pages)


@functools.lru_cache(maxsize=1024)
def _append_plan(layouts):
    """(dims, their reference, dtype code, device) of a fab_paged_append call on
    q, k, v, wq, wk, cos, sin, starts, lens, table, k_cache, v_cache."""
    q, k, v, wq, wk, cos, sin, starts, lens, table, k_cache, v_cache = layouts
    if len(q[0]) != 3 or len(k[0]) != 3 or len(v[0]) != 3:
        raise ValueError("q, k, v must be 3-D: (T,H,DK), (T,Hkv,DK), (T,Hkv,DV)")
    T, H, DK = q[0]
    dt = q[2]
    code, dev = _code(dt), _one_device(layouts)
    dims = _paged_dims(H, T, dt, k_cache, v_cache, starts, lens, table)
    dims.rot, dims.P = _tables(cos, sin, wq, wk, DK, dt)
    dims.ldq = _ld(q, "q", dt, (T, H, dims.DK))
    dims.ldk = _ld(k, "k", dt, (T, dims.Hkv, DK))
    dims.ldv = _ld(v, "v", dt, (T, dims.Hkv, dims.DV))
    return dims, ctypes.byref(dims), code, dev


def _append_call(plan, q, k, v, wq, wk, cos, sin, eps, interleaved, starts, lens, table, q_out, k_cache, v_cache,
                 stream):
    dev = plan[3]
    _current(dev)
    _check(lib().fab_paged_append(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _addr(wq), _addr(wk), _addr(cos), _addr(sin), eps,
        1 if interleaved else 0, starts.data_ptr(), lens.data_ptr(), table.data_ptr(), plan[2], plan[1],
        q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _raw_stream(stream, dev)), "fab_paged_append")


def fab_paged_append(q, k, v, wq, wk, cos, sin, eps, interleaved, starts, lens, table, q_out, k_cache, v_cache,
                     stream=None):
    plan = _append_plan(_layouts(q, k, v, wq, wk, cos, sin, starts, lens, table, k_cache, v_cache))
    _outputs(plan[3], (q_out, "q_out", q.dtype, q.shape))
    _append_call(plan, q, k, v, wq, wk, cos, sin, eps, interleaved, starts, lens, table, q_out, k_cache, v_cache,
                 stream)


def fab_paged_attention_workspace_bytes(dims: fab_paged_dims, dtype: int) -> int:
    return lib().fab_paged_attention_workspace_bytes(ctypes.byref(dims), int(dtype))


@functools.lru_cache(maxsize=1024)
def _paged_plan(layouts):
    """(dims, their reference, dtype code, device, workspace bytes) of a
    fab_paged_attention call on q, k_cache, v_cache, starts, lens, table."""
    q, k_cache, v_cache, starts, lens, table = layouts
    if len(q[0]) != 3:
        raise ValueError("q must be 3-D: (T,H,DK)")
    T, H, DK = q[0]
    dt = q[2]
    code, dev = _code(dt), _one_device(layouts)
    dims = _paged_dims(H, T, dt, k_cache, v_cache, starts, lens, table)
    _whole(q, "q", dt, (T, H, dims.DK))
    _current(dev)  # (the workspace's size goes by the current device)
    return dims, ctypes.byref(dims), code, dev, fab_paged_attention_workspace_bytes(dims, code)


def _paged_call(plan, q, k_cache, v_cache, starts, lens, table, causal, scale, ws, wsb, o, lse, stream):
    dev = plan[3]
    _current(dev)
    _check(lib().fab_paged_attention(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), starts.data_ptr(), lens.data_ptr(), table.data_ptr(),
        1 if causal else 0, float(scale), plan[2], plan[1], _addr(ws), wsb, o.data_ptr(), _addr(lse),
        _raw_stream(stream, dev)), "fab_paged_attention")


def fab_paged_attention(q, k_cache, v_cache, starts, lens, table, causal, scale, workspace, o, lse, stream=None):
    """lse may be None, and workspace where its size is 0."""
    plan = _paged_plan(_layouts(q, k_cache, v_cache, starts, lens, table))
    T, H = q.shape[:2]
    _outputs(plan[3], (o, "o", q.dtype, (T, H, plan[0].DV)), (lse, "lse", torch.float32, (H, T)))
    _paged_call(plan, q, k_cache, v_cache, starts, lens, table, causal, scale, workspace, _bytes(workspace, plan[3]), o,
                lse, stream)


def _on(stream):
    """A context whose allocations belong to `stream` (None: the current one),
    so that torch does not hand their memory to other work too early."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def qk_norm_rope(q, k, v, wq=None, wk=None, cos=None, sin=None, pos=None, eps=1e-6, interleaved=False, stream=None):
    """Projection rows q (B,N,H,DK), k (B,N,Hkv,DK), v (B,N,Hkv,DV) or None to
    what forward() takes: q (B,H,N,DK), k (B,Hkv,N,DK) normalised per head
    (where weights are given) and rotated (where tables are), v (B,Hkv,N,DV)."""
    plan = _rope_plan(_layouts(q, k, v, wq, wk, cos, sin, pos))
    with _on(stream):
        B, N, H, DK = q.shape
        dt, dev = q.dtype, q.device
        qo = torch.empty((B, H, N, DK), dtype=dt, device=dev)
        ko = torch.empty((B, k.shape[2], N, DK), dtype=dt, device=dev)
        vo = None if v is None else torch.empty((B, v.shape[2], N, v.shape[3]), dtype=dt, device=dev)
        _rope_call(plan, q, k, v, wq, wk, cos, sin, pos, eps, interleaved, qo, ko, vo, stream)
    return qo, ko, vo


def qk_norm_rope_backward(dq, dk, dv, q, k, wq=None, wk=None, cos=None, sin=None, pos=None, eps=1e-6,
                          interleaved=False, dtype=None, stream=None):
    """The gradients of qk_norm_rope's q, k, v, wq, wk for those of its results
    (unpack()'s float32 slices): (gq (B,N,H,DK), gk (B,N,Hkv,DK), gv (B,N,Hkv,DV)
    or None, gwq, gwk float32 (DK,) or None).  gq, gk and gv are in `dtype`
    (None: q's) and are views of one row of H*DK + Hkv*DK + Hkv*DV values a
    token: gq._base is the gradient of a fused projection."""
    dtype = q.dtype if dtype is None else dtype
    plan = _rope_backward_plan(_layouts(dq, dk, dv, q, k, wq, wk, cos, sin, pos), dtype, None)
    B, H, N, DK = dq.shape
    Hkv, row, dev = dk.shape[1], plan[0].ldgq, dq.device
    with _on(stream):
        g = torch.empty((B, N, row), dtype=dtype, device=dev)
        gq = g.as_strided((B, N, H, DK), (N * row, row, DK, 1))
        gk = g.as_strided((B, N, Hkv, DK), (N * row, row, DK, 1), H * DK)
        gv = None
        if dv is not None:
            DV = dv.shape[3]
            gv = g.as_strided((B, N, Hkv, DV), (N * row, row, DV, 1), (H + Hkv) * DK)
        gwq = None if wq is None else torch.empty((DK,), dtype=torch.float32, device=dev)
        gwk = None if wk is None else torch.empty((DK,), dtype=torch.float32, device=dev)
        ws, wsb = None, 0
        if wq is not None or wk is not None:
            wsb = plan[4]
            ws = torch.empty((wsb,), dtype=torch.uint8, device=dev)
        _rope_backward_call(plan, dq, dk, dv, q, k, wq, wk, cos, sin, pos, eps, interleaved, ws, wsb, gq, gk, gv, gwq,
                            gwk, stream)
    return gq, gk, gv, gwq, gwk


def paged_append(q, k, v, wq, wk, cos, sin, starts, lens, table, k_cache, v_cache, eps=1e-6, interleaved=False,
                 stream=None):
    """Puts the new tokens' keys and values into the caches and returns their
    queries (T,H,DK), normalised and rotated as qk_norm_rope does; rows of
    padding tokens are left as allocated."""
    plan = _append_plan(_layouts(q, k, v, wq, wk, cos, sin, starts, lens, table, k_cache, v_cache))
    with _on(stream):
        qo = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _append_call(plan, q, k, v, wq, wk, cos, sin, eps, interleaved, starts, lens, table, qo, k_cache, v_cache,
                     stream)
    return qo


def alloc_paged(q, k_cache, v_cache, table):
    """A workspace (uint8 tensor) for fab_paged_attention calls of these sizes."""
    pages, Hkv, page, DK = k_cache.shape
    B, max_pages = table.shape
    dims = fab_paged_dims(B, q.shape[0], q.shape[1], Hkv, DK, v_cache.shape[3], page, pages, max_pages)
    wsb = fab_paged_attention_workspace_bytes(dims, dtype_code(q))
    return torch.empty(wsb, dtype=torch.uint8, device=q.device)


def paged_attention(q, k_cache, v_cache, starts, lens, table, causal=True, scale=None, stream=None):
    """Returns (o (T,H,DV) in q's dtype, lse (H,T) float32); rows of padding
    tokens are left as allocated."""
    plan = _paged_plan(_layouts(q, k_cache, v_cache, starts, lens, table))
    T, H, DK = q.shape
    scale = DK ** -0.5 if scale is None else scale
    with _on(stream):
        dev, wsb = q.device, plan[4]
        o = torch.empty((T, H, v_cache.shape[3]), dtype=q.dtype, device=dev)
        lse = torch.empty((H, T), dtype=torch.float32, device=dev)
        ws = torch.empty((wsb,), dtype=torch.uint8, device=dev) if wsb > 0 else None
        _paged_call(plan, q, k_cache, v_cache, starts, lens, table, causal, scale, ws, wsb, o, lse, stream)
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

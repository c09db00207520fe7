"""Python binding of libcq (include/cq.h, include/cq_kv.h): argument marshalling only.

The raw functions carry the C names and arguments (integers for pointers and
the stream) and return the integer cq_status. The ``*_t`` helpers take torch
CUDA tensors, allocate outputs with torch, call the C function on the current
stream and raise ``CqError`` on a non-zero status. Every step of the
computation runs in libcq's CUDA kernels; there is no other path. Importing
this module does not need a GPU; calling it does, and a missing libcq.so is
an error, never a fallback.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libcq.so")

Q4_0, Q4_1, Q8_0, Q8_1, Q4_K, Q5_K, Q6_K, Q8_K = 2, 3, 8, 9, 12, 13, 14, 15
ACT_FOR = {Q4_0: Q8_0, Q8_0: Q8_0, Q4_1: Q8_1, Q4_K: Q8_K, Q5_K: Q8_K, Q6_K: Q8_K}
BLOCK = {Q4_0: (32, 18), Q4_1: (32, 20), Q8_0: (32, 34), Q8_1: (32, 36), Q4_K: (256, 144), Q5_K: (256, 176),
         Q6_K: (256, 210), Q8_K: (256, 292)}
FMT = {"q4_0": Q4_0, "q4_1": Q4_1, "q8_0": Q8_0, "q8_1": Q8_1, "q4_k": Q4_K, "q5_k": Q5_K, "q6_k": Q6_K,
       "q8_k": Q8_K}

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_FORMAT, ERR_SHAPE, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_CUDA, \
    ERR_DEVICE_STATUS, ERR_TIMEOUT = range(9)
DEV_BAD_EXPERT_ID, DEV_DUP_EXPERT_ID, DEV_WAIT_TIMEOUT = 0x1, 0x2, 0x4
DEV_KV_LENGTH, DEV_KV_BLOCKS, DEV_KV_PAGES, DEV_KV_TOKENS, DEV_KV_PAGE = 0x08, 0x10, 0x20, 0x40, 0x80
ATTN_WORKSPACE_ZERO = 4096     # bytes of an attention workspace that are zero before its first use
F32, F16, BF16 = 0, 1, 30      # value types of keys, values and queries (cq_dtype)

# Every symbol include/cq.h and include/cq_kv.h declare, with (restype, argtypes).
_P, _I64, _I, _SZ, _F = C.c_void_p, C.c_int64, C.c_int, C.c_size_t, C.c_float
SIGNATURES = {
    "cq_quantize_act": (_I, [_I, _I64, _I64, _P, _P, _P]),
    "cq_gemv": (_I, [_I, _I64, _I64, _I64, _P, _P, _P, _P]),
    "cq_gemv_x": (_I, [_I, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "cq_gemv_swiglu": (_I, [_I, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "cq_gemm": (_I, [_I, _I64, _I64, _I64, _P, _P, _P, _P]),
    "cq_gemm_noalloc": (_I, [_I, _I64, _I64, _I64, _P, _P, _P, _P]),
    "cq_gemm_workspace_size": (_SZ, [_I, _I64, _I64, _I64]),
    "cq_gemm_ws": (_I, [_I, _I64, _I64, _I64, _P, _P, _P, _P, _SZ, _P]),
    "cq_moe_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
    "cq_moe_gemv": (_I, [_I, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "cq_moe_gemv_noalloc": (_I, [_I, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P]),
    "cq_moe_workspace_offsets": (_I, [_I64, _I64, _I64, _I64, _I64, _P, _P, _P]),
    "cq_moe_read_status": (_I, [_P, _P, _P]),
    "cq_moe_noalloc_read_status": (_I, [_P, _P]),
    "cq_read_device_status": (_I, [_P, _P, _P]),
    "cq_read_global_status": (_I, [_P, _I]),
    "cq_status_string": (C.c_char_p, [_I]),
    "cq_set_option": (_I, [_I, _I64]),
    "cq_selftest_wait_timeout": (_I, [_I64, _P, _P]),
    "cq_repack_size": (_SZ, [_I, _I64, _I64]),
    "cq_repack": (_I, [_I, _I64, _I64, _P, _P, _P]),
    "cq_gemv_packed": (_I, [_I, _I64, _I64, _I64, _P, _P, _P, _P]),
    "cq_kv_plan": (_I, [_I64, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P]),
    "cq_kv_append": (_I, [_P, _I, _I64, _P, _I64, _P, _I64, _P, _P]),
    "cq_kv_read": (_I, [_P, _I, _I64, _P, _P, _P, _P]),
    "cq_attn_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "cq_attn_paged": (_I, [_P, _I, _I64, _I64, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _P, _F, _I, _I64, _P, _I64, _P,
                           _P, _SZ, _P]),
}


class cq_kv_cache(C.Structure):
    """The C struct of an 8-bit paged key/value cache (include/cq_kv.h)."""
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("num_pages", _I64), ("page_stride", _I64),
                ("scale_stride", _I64), ("page_size", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32),
                ("reserved", C.c_int32)]


OPT_WEIGHTS_CONST = 1

_lock = threading.Lock()
_lib = None


class CqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


def lib(path: str | None = None):
    """Load libcq.so (once). Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None or path is not None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"{p} is missing: build it with `python -m gemm_gguf_block_gb300.build`")
            L = C.CDLL(p)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype, f.argtypes = res, args
            if path is not None:
                return L
            _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().cq_status_string(s).decode()


# ------------------------------------------------------------------ raw C calls
def cq_quantize_act(act_fmt, M, K, x, xq, stream=0):
    return lib().cq_quantize_act(act_fmt, M, K, x, xq, stream)


def cq_gemv(w_fmt, M, N, K, W, xq, y, stream=0):
    return lib().cq_gemv(w_fmt, M, N, K, W, xq, y, stream)


def cq_gemv_x(w_fmt, M, N, K, W, x, xq, y, stream=0):
    return lib().cq_gemv_x(w_fmt, M, N, K, W, x, xq, y, stream)


def cq_gemv_swiglu(w_fmt, M, F, K, W_gate, W_up, xq, h, stream=0):
    return lib().cq_gemv_swiglu(w_fmt, M, F, K, W_gate, W_up, xq, h, stream)


def cq_gemm(w_fmt, M, N, K, W, xq, y, stream=0):
    return lib().cq_gemm(w_fmt, M, N, K, W, xq, y, stream)


def cq_gemm_noalloc(w_fmt, M, N, K, W, xq, y, stream=0):
    return lib().cq_gemm_noalloc(w_fmt, M, N, K, W, xq, y, stream)


def cq_selftest_wait_timeout(limit_ns, stream=0):
    """(status, device code) of the bounded-wait self-test."""
    code = C.c_int32(0)
    st = lib().cq_selftest_wait_timeout(limit_ns, C.byref(code), stream)
    return st, code.value


def cq_set_option(opt, value):
    return lib().cq_set_option(opt, value)


def cq_repack_size(w_fmt, N, K):
    return lib().cq_repack_size(w_fmt, N, K)


def cq_repack(w_fmt, N, K, W, Wp, stream=0):
    return lib().cq_repack(w_fmt, N, K, W, Wp, stream)


def cq_gemv_packed(w_fmt, M, N, K, Wp, xq, y, stream=0):
    return lib().cq_gemv_packed(w_fmt, M, N, K, Wp, xq, y, stream)


def cq_kv_plan(R, page_size, max_blocks, num_pages, past_len, new_len, free_pages, n_free, block_table, T, kv_len,
               q_start, slots, positions, used, stream=0):
    return lib().cq_kv_plan(R, page_size, max_blocks, num_pages, past_len, new_len, free_pages, n_free, block_table, T,
                            kv_len, q_start, slots, positions, used, stream)


def cq_kv_append(cache, dtype, T, k, k_stride, v, v_stride, slots, stream=0):
    """cache: the address of a cq_kv_cache (ctypes.addressof), as in the calls below."""
    return lib().cq_kv_append(cache, dtype, T, k, k_stride, v, v_stride, slots, stream)


def cq_kv_read(cache, dtype, T, slots, k_out, v_out, stream=0):
    return lib().cq_kv_read(cache, dtype, T, slots, k_out, v_out, stream)


def cq_attn_workspace_size(q_heads, kv_heads, head_dim):
    return lib().cq_attn_workspace_size(q_heads, kv_heads, head_dim)


def cq_attn_paged(cache, dtype, R, T, q_heads, max_new, max_kv, q, q_stride, block_table, max_blocks, kv_len, q_start,
                  scale, causal, window, out, out_stride, lse, ws, ws_bytes, stream=0):
    return lib().cq_attn_paged(cache, dtype, R, T, q_heads, max_new, max_kv, q, q_stride, block_table, max_blocks,
                               kv_len, q_start, scale, causal, window, out, out_stride, lse, ws, ws_bytes, stream)


def cq_gemm_workspace_size(w_fmt, M, N, K):
    return lib().cq_gemm_workspace_size(w_fmt, M, N, K)


def cq_gemm_ws(w_fmt, M, N, K, W, xq, y, ws, ws_bytes, stream=0):
    return lib().cq_gemm_ws(w_fmt, M, N, K, W, xq, y, ws, ws_bytes, stream)


def cq_moe_workspace_size(T, K, F, E, topk):
    return lib().cq_moe_workspace_size(T, K, F, E, topk)


def cq_moe_gemv(w_fmt, T, K, F, E, topk, W_gate, W_up, W_down, ids, route_w, xq, y, ws, ws_bytes, stream=0):
    return lib().cq_moe_gemv(w_fmt, T, K, F, E, topk, W_gate, W_up, W_down, ids, route_w, xq, y, ws,
                             ws_bytes, stream)


def cq_moe_gemv_noalloc(w_fmt, T, K, F, E, topk, W_gate, W_up, W_down, ids, route_w, xq, y, stream=0):
    """Routed FFN without a caller workspace (scratch in a fixed device array of the library)."""
    return lib().cq_moe_gemv_noalloc(w_fmt, T, K, F, E, topk, W_gate, W_up, W_down, ids, route_w, xq, y, stream)


def cq_moe_workspace_offsets(T, K, F, E, topk):
    a, b, c = C.c_size_t(), C.c_size_t(), C.c_size_t()
    st = lib().cq_moe_workspace_offsets(T, K, F, E, topk, C.addressof(a), C.addressof(b), C.addressof(c))
    return st, a.value, b.value, c.value


def cq_moe_read_status(ws, stream=0):
    code = C.c_int32()
    st = lib().cq_moe_read_status(ws, C.addressof(code), stream)
    return st, code.value


def cq_moe_noalloc_read_status(stream=0):
    code = C.c_int32()
    st = lib().cq_moe_noalloc_read_status(C.addressof(code), stream)
    return st, code.value


def cq_read_device_status(ws=None, stream=0):
    """(status, code) of a MoE workspace's status word, or (ws None) of the library's own word."""
    code = C.c_int32()
    st = lib().cq_read_device_status(ws, C.addressof(code), stream)
    return st, code.value


def cq_read_global_status(clear=1):
    code = C.c_int32()
    st = lib().cq_read_global_status(C.addressof(code), clear)
    return st, code.value


# --------------------------------------------------------- torch conveniences
def _torch():
    import torch
    return torch


def _stream_handle():
    return _torch().cuda.current_stream().cuda_stream


def row_bytes(fmt: int, K: int) -> int:
    e, b = BLOCK[fmt]
    return K // e * b


def _check(fn, st):
    if st != OK:
        raise CqError(fn, st)


def quantize_act_t(x, act_fmt: int):
    """x: CUDA fp32 [M, K] -> uint8 [M, row_bytes(act_fmt, K)]."""
    torch = _torch()
    M, K = x.shape
    xq = torch.empty((M, row_bytes(act_fmt, K)), dtype=torch.uint8, device=x.device)
    _check("cq_quantize_act", cq_quantize_act(act_fmt, M, K, x.data_ptr(), xq.data_ptr(), _stream_handle()))
    return xq


def gemv_t(W, xq, w_fmt: int, K: int, out=None):
    """W: uint8 [N, row_bytes]; xq: uint8 [M, act_row_bytes] (M <= 16) -> fp32 [M, N]."""
    torch = _torch()
    N, M = W.shape[0], xq.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=W.device)
    _check("cq_gemv", cq_gemv(w_fmt, M, N, K, W.data_ptr(), xq.data_ptr(), y.data_ptr(), _stream_handle()))
    return y


def repack_t(W, w_fmt: int, K: int):
    """cq_repack: W uint8 [N, row_bytes] -> the packed layout, uint8 [cq_repack_size]."""
    torch = _torch()
    N = W.shape[0]
    size = cq_repack_size(w_fmt, N, K)
    if size == 0 and N > 0:
        raise CqError("cq_repack_size", ERR_SHAPE)
    Wp = torch.empty(size, dtype=torch.uint8, device=W.device)
    _check("cq_repack", cq_repack(w_fmt, N, K, W.data_ptr(), Wp.data_ptr(), _stream_handle()))
    return Wp


def gemv_packed_t(Wp, xq, w_fmt: int, N: int, K: int, out=None):
    """cq_gemv_packed: Wp from repack_t; xq uint8 [M, act_row_bytes] (M <= 16) -> fp32 [M, N]."""
    torch = _torch()
    M = xq.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=Wp.device)
    _check("cq_gemv_packed", cq_gemv_packed(w_fmt, M, N, K, Wp.data_ptr(), xq.data_ptr(), y.data_ptr(),
                                            _stream_handle()))
    return y


def gemv_x_t(W, x, w_fmt: int, out=None):
    """cq_gemv_x: x fp32 [M, K] (M <= 16) -> (y fp32 [M, N], xq uint8 [M, act_row_bytes])."""
    torch = _torch()
    M, K = x.shape
    N = W.shape[0]
    xq = torch.empty((M, row_bytes(ACT_FOR[w_fmt], K)), dtype=torch.uint8, device=x.device)
    y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=x.device)
    _check("cq_gemv_x", cq_gemv_x(w_fmt, M, N, K, W.data_ptr(), x.data_ptr(), xq.data_ptr(), y.data_ptr(),
                                  _stream_handle()))
    return y, xq


def gemv_swiglu_t(Wg, Wu, xq, w_fmt: int, K: int, out=None):
    """cq_gemv_swiglu: Wg, Wu uint8 [F, row_bytes]; xq uint8 [M, act_row_bytes] (M <= 16)
    -> h fp32 [M, F] = silu(Wg . x) * (Wu . x)."""
    torch = _torch()
    F, M = Wg.shape[0], xq.shape[0]
    h = out if out is not None else torch.empty((M, F), dtype=torch.float32, device=Wg.device)
    _check("cq_gemv_swiglu", cq_gemv_swiglu(w_fmt, M, F, K, Wg.data_ptr(), Wu.data_ptr(), xq.data_ptr(),
                                            h.data_ptr(), _stream_handle()))
    return h


def gemm_t(W, xq, w_fmt: int, K: int, out=None):
    torch = _torch()
    N, M = W.shape[0], xq.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=W.device)
    _check("cq_gemm", cq_gemm(w_fmt, M, N, K, W.data_ptr(), xq.data_ptr(), y.data_ptr(), _stream_handle()))
    return y


def gemm_noalloc_t(W, xq, w_fmt: int, K: int, out=None):
    torch = _torch()
    N, M = W.shape[0], xq.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=W.device)
    _check("cq_gemm_noalloc", cq_gemm_noalloc(w_fmt, M, N, K, W.data_ptr(), xq.data_ptr(), y.data_ptr(),
                                              _stream_handle()))
    return y


def gemm_ws_t(W, xq, w_fmt: int, K: int, ws=None, out=None):
    """cq_gemm_ws with a workspace tensor (allocated here when not given)."""
    torch = _torch()
    N, M = W.shape[0], xq.shape[0]
    need = cq_gemm_workspace_size(w_fmt, M, N, K)
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=W.device)
    y = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=W.device)
    _check("cq_gemm_ws", cq_gemm_ws(w_fmt, M, N, K, W.data_ptr(), xq.data_ptr(), y.data_ptr(), ws.data_ptr(),
                                    ws.numel(), _stream_handle()))
    return y


def moe_t(W_gate, W_up, W_down, ids, route_w, xq, K: int, F: int, ws=None, out=None):
    """Routed FFN. Returns (y [T, K] fp32, workspace uint8 tensor)."""
    torch = _torch()
    E = W_gate.shape[0]
    T, topk = ids.shape
    need = cq_moe_workspace_size(T, K, F, E, topk)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=xq.device)
    y = out if out is not None else torch.empty((T, K), dtype=torch.float32, device=xq.device)
    _check("cq_moe_gemv", cq_moe_gemv(Q4_0, T, K, F, E, topk, W_gate.data_ptr(), W_up.data_ptr(),
                                      W_down.data_ptr(), ids.data_ptr(), route_w.data_ptr(), xq.data_ptr(),
                                      y.data_ptr(), ws.data_ptr(), ws.numel(), _stream_handle()))
    return y, ws


# ------------------------------------------------- 8-bit paged key/value cache
# These calls are made once a layer and step, on small batches too, so the
# helpers look at each tensor once and keep what does not change.
_tables = {}


def _torch_tables():
    """torch, its integer types, the cq_dtype of each value type, the current device and the raw stream of a device."""
    if not _tables:
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda d: torch.cuda.current_stream(d).cuda_stream)
        _tables["all"] = (torch, torch.int32, torch.int64,
                          {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}, raw)
    return _tables["all"]


def _stream_of(fn, raw, i, *tensors):
    """The current stream of device i. A call whose tensors are on the host, or not all on that device, is refused here:
    the library gets their addresses only."""
    if i < 0:
        raise CqError(fn, ERR_INVALID_ARG)
    for t in tensors:
        if t.get_device() != i:
            raise CqError(fn, ERR_INVALID_ARG)
    return raw(i)


def _rows(fn, t, width):
    """Pointer, row stride (elements) and rows of [T, width] or [T, heads, head_dim] with contiguous rows."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        ok = shape[1] * shape[2] == width and stride[2] == 1 and (shape[1] == 1 or stride[1] == shape[2])
    else:
        ok = len(shape) == 2 and shape[1] == width and stride[1] == 1
    if not ok:
        raise CqError(fn, ERR_SHAPE)
    T = shape[0]
    return t.data_ptr(), stride[0] if T > 1 else width, T


def _vec(fn, t, dtype, n):
    """Pointer of a contiguous vector of this type and length."""
    shape = t.shape
    if t.dtype != dtype or len(shape) != 1 or shape[0] != n or not t.is_contiguous():
        raise CqError(fn, ERR_SHAPE)
    return t.data_ptr()


def _table(fn, t, i32, R):
    """Pointer and width of a contiguous int32 block table of R rows."""
    shape = t.shape
    if t.dtype != i32 or len(shape) != 2 or shape[0] != R or not t.is_contiguous():
        raise CqError(fn, ERR_SHAPE)
    return t.data_ptr(), shape[1]


class KVCache:
    """An 8-bit paged key/value cache over the caller's tensors: k, v int8 [pages, kv heads, page tokens, head size]
    (pages may be strided: halves of one allocation), k_scale, v_scale fp32 [pages, kv heads]."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "num_pages", "kv_heads", "page_size", "head_dim", "device", "_c", "addr")

    def __init__(self, k, v, k_scale, v_scale):
        torch = _torch()
        if k.dim() != 4 or v.shape != k.shape or k.dtype != torch.int8 or v.dtype != torch.int8 or \
                v.stride() != k.stride() or k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or \
                k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2] or k_scale.stride() != v_scale.stride():
            raise CqError("cq_kv_cache", ERR_SHAPE)
        n, h, p, d = k.shape
        if k.stride()[1:] != (p * d, d, 1) or (h > 1 and k_scale.stride(1) != 1):
            raise CqError("cq_kv_cache", ERR_SHAPE)
        self.device = k.get_device()                     # -1 on the host: the calls refuse it
        if any(t.get_device() != self.device for t in (v, k_scale, v_scale)):
            raise CqError("cq_kv_cache", ERR_INVALID_ARG)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = n, h, p, d
        one = n <= 1     # a single page's strides say nothing
        self._c = cq_kv_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), n,
                              h * p * d if one else k.stride(0), h if one else k_scale.stride(0), p, h, d, 0)
        self.addr = C.addressof(self._c)

    @classmethod
    def empty(cls, num_pages, kv_heads, page_size, head_dim, device="cuda"):
        """A new cache; its pages hold nothing until they are written."""
        torch = _torch()
        kv = torch.zeros((2, num_pages, kv_heads, page_size, head_dim), dtype=torch.int8, device=device)
        sc = torch.zeros((2, num_pages, kv_heads), dtype=torch.float32, device=device)
        return cls(kv[0], kv[1], sc[0], sc[1])


def kv_plan_t(past_len, new_len, block_table, free_pages, page_size: int, num_pages: int, tokens: int):
    """cq_kv_plan: int32 past_len, new_len [R], block_table [R, max_blocks] (updated in place), free_pages [n]
    -> kv_len int32 [R], q_start int32 [R + 1], slots int64 [tokens], positions int32 [tokens], used int32 [2]."""
    torch, i32, i64, _, raw = _torch_tables()
    fn, R, n_free = "cq_kv_plan", past_len.shape[0], free_pages.shape[0]
    tp, wide = _table(fn, block_table, i32, R)
    past, new, free = _vec(fn, past_len, i32, R), _vec(fn, new_len, i32, R), _vec(fn, free_pages, i32, n_free)
    stream = _stream_of(fn, raw, past_len.get_device(), new_len, block_table, free_pages)
    dev = past_len.device
    # (an allocation each costs the host less than views of one)
    kv_len, q_start = torch.empty(R, dtype=i32, device=dev), torch.empty(R + 1, dtype=i32, device=dev)
    slots, positions = torch.empty(tokens, dtype=i64, device=dev), torch.empty(tokens, dtype=i32, device=dev)
    used = torch.empty(2, dtype=i32, device=dev)
    st = (_lib or lib()).cq_kv_plan(R, page_size, wide, num_pages, past, new, free, n_free, tp, tokens,
                                    kv_len.data_ptr(), q_start.data_ptr(), slots.data_ptr(), positions.data_ptr(),
                                    used.data_ptr(), stream)
    if st:
        raise CqError(fn, st)
    return kv_len, q_start, slots, positions, used


def kv_append_t(cache: KVCache, k, v, slots):
    """cq_kv_append: k, v [T, heads * size] or [T, heads, size] (fp32, fp16 or bf16, rows may be strided), slots int64 [T]."""
    _, _, i64, dtypes, raw = _torch_tables()
    fn, width, dt = "cq_kv_append", cache.kv_heads * cache.head_dim, k.dtype
    kp, ks, T = _rows(fn, k, width)
    vp, vs, Tv = _rows(fn, v, width)
    if Tv != T or v.dtype != dt:
        raise CqError(fn, ERR_SHAPE)
    st = (_lib or lib()).cq_kv_append(cache.addr, dtypes.get(dt, -1), T, kp, ks, vp, vs, _vec(fn, slots, i64, T),
                                      _stream_of(fn, raw, cache.device, k, v, slots))
    if st:
        raise CqError(fn, st)


def kv_read_t(cache: KVCache, slots, dtype=None):
    """cq_kv_read: slots int64 [T] -> keys and values [T, heads, size] of `dtype` (fp32 by default)."""
    torch, _, i64, dtypes, raw = _torch_tables()
    fn, T = "cq_kv_read", slots.shape[0]
    sp, stream = _vec(fn, slots, i64, T), _stream_of(fn, raw, cache.device, slots)
    dt = dtype or torch.float32
    if dt not in dtypes:
        raise CqError(fn, ERR_UNSUPPORTED_FORMAT)
    shape, dev = (T, cache.kv_heads, cache.head_dim), slots.device
    k, v = torch.empty(shape, dtype=dt, device=dev), torch.empty(shape, dtype=dt, device=dev)
    st = (_lib or lib()).cq_kv_read(cache.addr, dtypes[dt], T, sp, k.data_ptr(), v.data_ptr(), stream)
    if st:
        raise CqError(fn, st)
    return k, v


def attn_workspace_t(q_heads: int, kv_heads: int, head_dim: int, device="cuda"):
    """A workspace for attn_paged_t, zeroed as its first use wants it (all of it: a fill of its beginning alone costs the
    host more than the device saves, 19 against 15 us)."""
    need = cq_attn_workspace_size(q_heads, kv_heads, head_dim)
    if need == 0:
        raise CqError("cq_attn_workspace_size", ERR_SHAPE)
    return _torch().zeros(need, dtype=_torch().uint8, device=device)


def attn_paged_t(q, cache: KVCache, block_table, kv_len, q_start, max_new: int, max_kv: int, *, scale=None,
                 causal: bool = True, window: int = 0, ws=None, out=None, lse=True):
    """cq_attn_paged: q [T, q heads, size] (fp32, fp16 or bf16; rows may be strided) over the cache
    -> (out [T, q heads, size], lse fp32 [T, q heads] or None). block_table int32 [R, max_blocks], kv_len int32 [R],
    q_start int32 [R + 1]; max_new: the most new tokens of any request (it chooses the kernels), max_kv: of kv_len (not
    used yet); scale 1 / sqrt(size) by default; ws: attn_workspace_t's, made here when not given;
    lse: a tensor, True for a new one, or None. Rows of no request (padding) are not written: undefined in new tensors."""
    torch, i32, _, dtypes, raw = _torch_tables()
    fn, D, dt = "cq_attn_paged", cache.head_dim, q.dtype
    shape = q.shape
    if len(shape) != 3 or shape[2] != D:
        raise CqError(fn, ERR_SHAPE)
    T, heads = shape[0], shape[1]
    R, width = kv_len.shape[0], heads * D
    qp, qs, _ = _rows(fn, q, width)
    tp, wide = _table(fn, block_table, i32, R)
    kvp, sp = _vec(fn, kv_len, i32, R), _vec(fn, q_start, i32, R + 1)
    stream, dev = _stream_of(fn, raw, cache.device, q, block_table, kv_len, q_start), q.device
    if ws is None:
        ws = attn_workspace_t(heads, cache.kv_heads, D, dev)
    elif ws.get_device() != cache.device or not ws.is_contiguous():
        raise CqError(fn, ERR_WORKSPACE)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=dev)
        op, os_ = out.data_ptr(), width
    else:
        op, os_, To = _rows(fn, out, width)
        if To != T or out.dtype != dt or out.get_device() != cache.device:
            raise CqError(fn, ERR_SHAPE)
    if lse is True:
        lse = torch.empty((T, heads), dtype=torch.float32, device=dev)
    elif lse is False:
        lse = None
    elif lse is not None and (lse.dtype != torch.float32 or lse.shape != (T, heads) or not lse.is_contiguous() or
                              lse.get_device() != cache.device):
        raise CqError(fn, ERR_SHAPE)
    st = (_lib or lib()).cq_attn_paged(cache.addr, dtypes.get(dt, -1), R, T, heads, max_new, max_kv, qp, qs, tp, wide,
                                       kvp, sp, D ** -0.5 if scale is None else scale, 1 if causal else 0, window, op,
                                       os_, None if lse is None else lse.data_ptr(), ws.data_ptr(),
                                       ws.numel() * ws.element_size(), stream)
    if st:
        raise CqError(fn, st)
    return out, lse

"""Fused-dequantisation GGUF quantized matmul for one GB300 (sm_103a).

A thin ctypes binding over libqmm.so, the C ABI declared in include/qmm.h.
It only marshals arguments: torch tensors supply device memory and the
current CUDA stream, and every step of the computation runs in the library's
CUDA kernels.  There is no CPU fallback: if libqmm.so is missing or cannot be
loaded, every call raises.

Names follow the C ABI (``qmm_gemv`` -> ``gemv`` and so on).  ``Matrix`` owns
a handle for a quantized weight tensor kept on the device.
"""
from __future__ import annotations

import ctypes
import os

Q8_0 = 8
Q4_K = 12
Q5_K = 13
Q6_K = 14
IQ4_NL = 20
F32, F16, BF16 = 0, 1, 30  # plain types (activations; F16, BF16 and Q8_0: a cache's types)

OK = 0
ERR_NULL, ERR_FORMAT, ERR_SHAPE, ERR_ALIGN, ERR_CUDA = -1, -2, -3, -4, -5
ERR_TIMEOUT, ERR_UNSUPPORTED, ERR_NOMEM, ERR_EXPERT, ERR_PAGE = -6, -7, -8, -9, -10

_HERE = os.path.dirname(os.path.abspath(__file__))
# QMM_LIBRARY may name another build of the library (e.g. an instrumented one).
LIB_PATH = os.environ.get("QMM_LIBRARY") or os.path.join(_HERE, "libqmm.so")
_lib = None

# Every entry point of include/qmm.h.
ENTRY_POINTS = (
    "qmm_create", "qmm_destroy", "qmm_gemv", "qmm_gemv_group", "qmm_gemv_batched",
    "qmm_moe_gemv", "qmm_swiglu", "qmm_moe_ffn", "qmm_gemm", "qmm_dequantize",
    "qmm_dequantize_bf16", "qmm_get_status", "qmm_last_error", "qmm_version",
    "qmm_gemv_noalloc", "qmm_gemm_group", "qmm_launch_count", "qmm_ffn_decode",
    "qmm_quantize_q8_k", "qmm_gemv_q8k", "qmm_gemv_q8k_group", "qmm_gemv_q8k_fused",
    "qmm_gemv_q8k_fused_group",
    "qmm_kv_create", "qmm_kv_bytes", "qmm_kv_destroy", "qmm_kv_append", "qmm_kv_read",
    "qmm_attn_decode", "qmm_kv_get_status", "qmm_logits_adjust",
)


class RopeDesc(ctypes.Structure):
    """qmm_rope."""
    _fields_ = [("n_rot", ctypes.c_int32), ("pairing", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4),
                ("inv_freq", ctypes.c_void_p)]


class AttnDesc(ctypes.Structure):
    """qmm_attn."""
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float),
                ("window", ctypes.c_int32), ("alibi", ctypes.c_void_p)]


class LogitRules(ctypes.Structure):
    """qmm_logit_rules."""
    _fields_ = [("history", ctypes.c_void_p), ("history_offsets", ctypes.c_void_p),
                ("n_history", ctypes.c_int64), ("repeat", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("frequency", ctypes.c_void_p),
                ("bias_ids", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("bias_offsets", ctypes.c_void_p), ("n_biases", ctypes.c_int64),
                ("mask", ctypes.c_void_p), ("ld_mask", ctypes.c_int64)]


class QmmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[{status}] {message}")
        self.status = status
        self.message = message


def lib() -> ctypes.CDLL:
    """The loaded libqmm.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m quantized_gguf_dequant_gb300.build` (there is no fallback)")
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
        sig = {
            "qmm_create": [i32, i64, i64, vp, ctypes.POINTER(vp)],
            "qmm_destroy": [vp],
            "qmm_gemv": [vp, vp, vp, vp],
            "qmm_gemv_group": [ctypes.POINTER(vp), i32, vp, ctypes.POINTER(vp), vp],
            "qmm_gemv_batched": [vp, vp, i64, i64, vp, i64, vp],
            "qmm_moe_gemv": [vp, i32, vp, i32, i32, vp, i32, vp, i32, vp, vp],
            "qmm_swiglu": [vp, vp, vp, i64, vp],
            "qmm_moe_ffn": [vp, vp, vp, i32, vp, i32, i32, vp, vp, i32, vp, vp],
            "qmm_gemm": [vp, vp, i64, vp, vp],
            "qmm_dequantize": [vp, i64, i64, vp, vp],
            "qmm_dequantize_bf16": [vp, i64, i64, vp, vp],
            "qmm_get_status": [vp],
            "qmm_last_error": [],
            "qmm_version": [],
            "qmm_gemv_noalloc": [i32, i64, i64, vp, vp, vp, vp],
            "qmm_gemm_group": [ctypes.POINTER(vp), i32, vp, i64, ctypes.POINTER(vp), vp],
            "qmm_ffn_decode": [vp, vp, vp, vp, vp, vp, vp],
            "qmm_quantize_q8_k": [vp, i64, vp, vp],
            "qmm_gemv_q8k": [vp, vp, vp, vp],
            "qmm_gemv_q8k_group": [ctypes.POINTER(vp), i32, vp, ctypes.POINTER(vp), vp],
            "qmm_gemv_q8k_fused": [vp, vp, vp, vp],
            "qmm_gemv_q8k_fused_group": [ctypes.POINTER(vp), i32, vp, ctypes.POINTER(vp), vp],
            "qmm_kv_create": [i32, i64, i32, i32, i32, vp, vp, ctypes.POINTER(vp)],
            "qmm_kv_bytes": [i32, i64, i32, i32, i32],
            "qmm_kv_destroy": [vp],
            "qmm_kv_append": [vp, i32, i64, vp, i64, vp, i64, vp, vp, i64, i32, vp, i64, vp,
                              ctypes.POINTER(RopeDesc), vp],
            "qmm_kv_read": [vp, i32, i64, vp, vp, i64, vp, i64, vp],
            "qmm_attn_decode": [vp, i32, i64, i32, vp, i64, vp, i64, vp,
                                ctypes.POINTER(AttnDesc), vp, i64, vp, vp],
            "qmm_kv_get_status": [vp],
            "qmm_logits_adjust": [i32, i64, i64, vp, i64, ctypes.POINTER(LogitRules), vp, i64,
                                  vp],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = i32
        L.qmm_last_error.restype = ctypes.c_char_p
        L.qmm_launch_count.argtypes = []
        L.qmm_launch_count.restype = ctypes.c_int64
        L.qmm_kv_bytes.restype = ctypes.c_int64
        _lib = L
    return _lib


def last_error() -> str:
    return lib().qmm_last_error().decode()


def version() -> int:
    return int(lib().qmm_version())


def launch_count() -> int:
    """Kernel launches the library has issued in this process so far."""
    return int(lib().qmm_launch_count())


def _check(rc: int):
    if rc != OK:
        raise QmmError(rc, last_error())


def _ptr(t) -> ctypes.c_void_p:
    if t is None:
        return ctypes.c_void_p(0)
    if isinstance(t, int):
        return ctypes.c_void_p(t)
    if not t.is_cuda:
        raise ValueError("tensor must live on the CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None) -> ctypes.c_void_p:
    import torch
    if stream is None:
        # the current stream's handle without building a Stream object
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return ctypes.c_void_p(raw(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


# --------------------------------------------------------------------- raw ABI

def create(fmt: int, N: int, K: int, w) -> int:
    h = ctypes.c_void_p()
    _check(lib().qmm_create(fmt, N, K, _ptr(w), ctypes.byref(h)))
    return h.value


def destroy(h: int):
    _check(lib().qmm_destroy(ctypes.c_void_p(h)))


def gemv(h: int, x, y, stream=None):
    _check(lib().qmm_gemv(ctypes.c_void_p(h), _ptr(x), _ptr(y), _stream(stream)))


def gemv_group(hs, x, ys, stream=None):
    n = len(hs)
    harr = (ctypes.c_void_p * n)(*[ctypes.c_void_p(h) for h in hs])
    yarr = (ctypes.c_void_p * n)(*[_ptr(y) for y in ys])
    _check(lib().qmm_gemv_group(harr, n, _ptr(x), yarr, _stream(stream)))


def gemv_batched(h: int, X, M: int, ldx: int, Y, ldy: int, stream=None):
    _check(lib().qmm_gemv_batched(ctypes.c_void_p(h), _ptr(X), M, ldx, _ptr(Y), ldy,
                                  _stream(stream)))


def moe_gemv(h: int, n_experts: int, ids, T: int, top_k: int, X, x_per_slot: int,
             route_w, Y, stream=None, route_on_input: bool = False):
    _check(lib().qmm_moe_gemv(ctypes.c_void_p(h), n_experts, _ptr(ids), T, top_k, _ptr(X),
                              int(x_per_slot), _ptr(route_w), int(route_on_input), _ptr(Y),
                              _stream(stream)))


def ffn_decode(hg: int, hu: int, hd: int, x, h, y, stream=None):
    """qmm_ffn_decode: h = silu(Wg x) * (Wu x), y = Wd h (one token)."""
    _check(lib().qmm_ffn_decode(ctypes.c_void_p(hg), ctypes.c_void_p(hu), ctypes.c_void_p(hd),
                                _ptr(x), _ptr(h), _ptr(y), _stream(stream)))


def swiglu(g, u, hout, n: int, stream=None):
    _check(lib().qmm_swiglu(_ptr(g), _ptr(u), _ptr(hout), n, _stream(stream)))


def moe_ffn(hg: int, hu: int, hd: int, n_experts: int, ids, T: int, top_k: int, X, route_w, Y,
            stream=None, route_on_input: bool = False):
    _check(lib().qmm_moe_ffn(ctypes.c_void_p(hg), ctypes.c_void_p(hu), ctypes.c_void_p(hd),
                             n_experts, _ptr(ids), T, top_k, _ptr(X), _ptr(route_w),
                             int(route_on_input), _ptr(Y), _stream(stream)))


Q8_K_BLOCK = 292  # bytes per 256 activations in the Q8_K encoding


def quantize_q8_k(x, K: int, xq, stream=None):
    """qmm_quantize_q8_k: K fp32 activations -> K/256 Q8_K blocks in xq."""
    _check(lib().qmm_quantize_q8_k(_ptr(x), K, _ptr(xq), _stream(stream)))


def gemv_q8k(h: int, xq, y, stream=None):
    """qmm_gemv_q8k: the integer-dot GEMV of a Q4_K matrix with Q8_K activations."""
    _check(lib().qmm_gemv_q8k(ctypes.c_void_p(h), _ptr(xq), _ptr(y), _stream(stream)))


def gemv_q8k_group(hs, xq, ys, stream=None):
    n = len(hs)
    harr = (ctypes.c_void_p * n)(*[ctypes.c_void_p(h) for h in hs])
    yarr = (ctypes.c_void_p * n)(*[_ptr(y) for y in ys])
    _check(lib().qmm_gemv_q8k_group(harr, n, _ptr(xq), yarr, _stream(stream)))


def gemv_q8k_fused(h: int, x, y, stream=None):
    """qmm_gemv_q8k_fused: the integer-dot GEMV on f32 activations, quantized
    to Q8_K inside the launch."""
    _check(lib().qmm_gemv_q8k_fused(ctypes.c_void_p(h), _ptr(x), _ptr(y), _stream(stream)))


def gemv_q8k_fused_group(hs, x, ys, stream=None):
    n = len(hs)
    harr = (ctypes.c_void_p * n)(*[ctypes.c_void_p(h) for h in hs])
    yarr = (ctypes.c_void_p * n)(*[_ptr(y) for y in ys])
    _check(lib().qmm_gemv_q8k_fused_group(harr, n, _ptr(x), yarr, _stream(stream)))


def gemm(h: int, X_bf16, M: int, Y, stream=None):
    _check(lib().qmm_gemm(ctypes.c_void_p(h), _ptr(X_bf16), M, _ptr(Y), _stream(stream)))


def gemm_group(hs, X_bf16, M: int, Ys, stream=None):
    n = len(hs)
    harr = (ctypes.c_void_p * n)(*[ctypes.c_void_p(h) for h in hs])
    yarr = (ctypes.c_void_p * n)(*[_ptr(y) for y in Ys])
    _check(lib().qmm_gemm_group(harr, n, _ptr(X_bf16), M, yarr, _stream(stream)))


def dequantize(h: int, row0: int, nrows: int, out, stream=None):
    _check(lib().qmm_dequantize(ctypes.c_void_p(h), row0, nrows, _ptr(out), _stream(stream)))


def dequantize_bf16(h: int, row0: int, nrows: int, out, stream=None):
    _check(lib().qmm_dequantize_bf16(ctypes.c_void_p(h), row0, nrows, _ptr(out),
                                     _stream(stream)))


def gemv_noalloc(fmt: int, N: int, K: int, w, x, y, stream=None):
    """qmm_gemv_noalloc: the decode GEMV without a handle or any device
    allocation (scratch lives in a fixed array inside the library)."""
    _check(lib().qmm_gemv_noalloc(fmt, N, K, _ptr(w), _ptr(x), _ptr(y), _stream(stream)))


def get_status(h: int) -> int:
    """The handle's device status (0 = OK); clears it."""
    return int(lib().qmm_get_status(ctypes.c_void_p(h)))


# --------------------------------------------------------------------- wrapper

class Matrix:
    """A quantized N x K matrix on the device (a torch uint8 tensor of its
    GGUF bytes) with its library handle."""

    def __init__(self, fmt: int, N: int, K: int, w_dev):
        import torch
        if w_dev.dtype != torch.uint8:
            raise ValueError("weights must be a uint8 tensor of GGUF block bytes")
        self.fmt, self.N, self.K = fmt, N, K
        self.w = w_dev  # keep the bytes alive as long as the handle
        self.h = create(fmt, N, K, w_dev)

    def close(self):
        if getattr(self, "h", None):
            destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def gemv(self, x, y=None, stream=None):
        import torch
        if y is None:
            y = torch.empty(self.N, dtype=torch.float32, device=x.device)
        gemv(self.h, x, y, stream)
        return y

    def gemv_batched(self, X, Y=None, stream=None):
        import torch
        M = X.shape[0]
        if Y is None:
            Y = torch.empty((M, self.N), dtype=torch.float32, device=X.device)
        gemv_batched(self.h, X, M, X.stride(0), Y, Y.stride(0), stream)
        return Y

    def gemm(self, X_bf16, Y=None, stream=None):
        import torch
        M = X_bf16.shape[0]
        if Y is None:
            Y = torch.empty((M, self.N), dtype=torch.float32, device=X_bf16.device)
        gemm(self.h, X_bf16, M, Y, stream)
        return Y

    def dequantize(self, row0=0, nrows=None, out=None, stream=None):
        import torch
        nrows = self.N - row0 if nrows is None else nrows
        if out is None:
            out = torch.empty((nrows, self.K), dtype=torch.float32, device=self.w.device)
        dequantize(self.h, row0, nrows, out, stream)
        return out

    def dequantize_bf16(self, row0=0, nrows=None, out=None, stream=None):
        import torch
        nrows = self.N - row0 if nrows is None else nrows
        if out is None:
            out = torch.empty((nrows, self.K), dtype=torch.int16, device=self.w.device)
        dequantize_bf16(self.h, row0, nrows, out, stream)
        return out

    def status(self) -> int:
        return get_status(self.h)


# ------------------------------------------------- the decode step around the products

_DTYPES = {}  # torch dtype -> plain type id, filled on first use


def _dtype(t) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16})
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{t.dtype} is not supported (float32, float16 and bfloat16 are)") from None


def _flat(t, name: str, dtype: str, n=None):
    """The pointer of a contiguous device tensor of the named dtype (and, with
    n given, of n elements); None stays None."""
    if t is None:
        return None
    if str(t.dtype) != "torch." + dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on the CUDA device")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements; {n} are needed")
    return t.data_ptr()


def _heads(t, name: str, T: int, heads: int, D: int, dtype=None):
    """(pointer, elements between tokens) of a [T, heads, D] tensor whose
    tokens may lie apart, such as a slice of a fused projection's output."""
    if t.dim() != 3 or tuple(t.shape) != (T, heads, D):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; {(T, heads, D)} is needed")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}; {dtype} is needed")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the CUDA device")
    s = t.stride()
    if s[2] != 1 or (heads > 1 and s[1] != D):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (s[0] if T > 1 else heads * D)


def _made_on(stream, *tensors):
    """Outputs allocated here for work on a stream that is not the current one
    must not return to the allocator before that work is done."""
    if stream is not None and not isinstance(stream, int):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


class Rope:
    """Rotary positions: inv_freq (fp32 on the device, one per pair), the pairs
    that turn by each axis (sections; default: one axis), and which dims are
    a pair: "halves" (i, i + n_rot/2) or "adjacent" (2i, 2i + 1)."""

    def __init__(self, inv_freq, sections=None, pairing: str = "halves"):
        n = inv_freq.numel()
        sections = [n] if sections is None else [int(x) for x in sections]
        if pairing not in ("halves", "adjacent"):
            raise ValueError(f"pairing {pairing!r}: 'halves' or 'adjacent'")
        if not 1 <= len(sections) <= 4 or sum(sections) != n:
            raise ValueError(f"sections {sections} must be 1 to 4 counts that sum to {n} pairs")
        self.inv_freq = inv_freq  # keep the device memory alive
        self.n_axes = len(sections)
        self.desc = RopeDesc(2 * n, int(pairing == "adjacent"), len(sections),
                             (ctypes.c_int32 * 4)(*sections),
                             _flat(inv_freq, "inv_freq", "float32"))


class KVCache:
    """A paged key-value cache on the device (qmm_kv_create) with the calls
    that use it.  kind: F16, BF16 or Q8_0.  k, v: its two buffers (any dtype,
    at least kv_bytes() bytes each); made and zeroed here when not given."""

    def __init__(self, kind: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
                 k=None, v=None):
        import torch
        self.kind, self.n_pages, self.page_size = kind, n_pages, page_size
        self.n_kv_heads, self.head_dim = n_kv_heads, head_dim
        need = kv_bytes(kind, n_pages, page_size, n_kv_heads, head_dim)
        if k is None:
            k = torch.zeros(need, dtype=torch.uint8, device="cuda")
        if v is None:
            v = torch.zeros(need, dtype=torch.uint8, device="cuda")
        for name, t in (("k", k), ("v", v)):
            if t.numel() * t.element_size() < need:
                raise ValueError(f"the {name} buffer holds {t.numel() * t.element_size()} bytes; "
                                 f"{need} are needed")
        self.k, self.v = k, v  # keep the buffers alive as long as the handle
        h = ctypes.c_void_p()
        _check(lib().qmm_kv_create(kind, n_pages, page_size, n_kv_heads, head_dim, _ptr(k),
                                   _ptr(v), ctypes.byref(h)))
        self.h = h.value

    def close(self):
        if getattr(self, "h", None):
            h, self.h = self.h, None
            _check(lib().qmm_kv_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def append(self, k, v, slots, q=None, pos=None, rope=None, q_out=None, stream=None):
        """qmm_kv_append: rotate q and k ([T, heads, head_dim]) and store k and
        v at slots ([T] int64).  pos: [n_axes, T] (or [T]) int32.  Returns the
        rotated q (into q_out, which may be q), or None without q."""
        import torch
        T, H, D = k.shape[0], self.n_kv_heads, self.head_dim
        kp, ldk = _heads(k, "k", T, H, D)
        vp, ldv = _heads(v, "v", T, H, D, k.dtype)
        sp = _flat(slots, "slots", "int64", T)
        qp = qop = None
        ldq = ldqo = n_q = 0
        if q is not None:
            n_q = q.shape[1]
            if q_out is None:
                q_out = torch.empty((T, n_q, D), dtype=q.dtype, device=q.device)
                _made_on(stream, q_out)
            qp, ldq = _heads(q, "q", T, n_q, D, k.dtype)
            qop, ldqo = _heads(q_out, "q_out", T, n_q, D, k.dtype)
        pp = desc = None
        if rope is not None:
            pp = _flat(pos, "pos", "int32", rope.n_axes * T)
            desc = ctypes.byref(rope.desc)
        _check(lib().qmm_kv_append(self.h, _dtype(k), T, kp, ldk, vp, ldv, sp, qp, ldq, n_q, qop,
                                   ldqo, pp, desc, _stream(stream)))
        return q_out if q is not None else None

    def attend(self, q, page_table, lens, scale=None, softcap: float = 0.0, window: int = 0,
               alibi=None, out=None, lse=None, return_lse: bool = False, stream=None):
        """qmm_attn_decode: attention of one new token of each sequence.  q:
        [n_seqs, n_q_heads, head_dim]; page_table: [n_seqs, pages] int32; lens:
        [n_seqs] int32; scale: 1/sqrt(head_dim) by default.  Returns out (like
        q), and with return_lse also lse ([n_seqs, n_q_heads] float32)."""
        import torch
        if q.dim() != 3:
            raise ValueError(f"q has shape {tuple(q.shape)}; [n_seqs, heads, head_dim] is needed")
        B, n_q, D = q.shape
        qp, ldq = _heads(q, "q", B, n_q, self.head_dim)
        if out is None:
            out = torch.empty((B, n_q, D), dtype=q.dtype, device=q.device)
            _made_on(stream, out)
        op, ldo = _heads(out, "out", B, n_q, D, q.dtype)
        if return_lse and lse is None:
            lse = torch.empty((B, n_q), dtype=torch.float32, device=q.device)
            _made_on(stream, lse)
        if page_table.dim() != 2 or page_table.shape[0] != B or page_table.stride(1) != 1 and \
                page_table.shape[1] > 1:
            raise ValueError(f"page_table must be [{B}, pages] with contiguous rows")
        if page_table.dtype != torch.int32 or not page_table.is_cuda:
            raise ValueError("page_table must be int32 on the CUDA device")
        width = page_table.shape[1]
        if B > 1 and page_table.stride(0) != width:
            page_table = page_table.contiguous()  # (the ABI takes a row's length as its stride)
            _made_on(stream, page_table)
        if scale is None:
            scale = D ** -0.5
        desc = AttnDesc(scale, softcap, window, _flat(alibi, "alibi", "float32", n_q))
        _check(lib().qmm_attn_decode(self.h, _dtype(q), B, n_q, qp, ldq, page_table.data_ptr(),
                                     width, _flat(lens, "lens", "int32", B), ctypes.byref(desc),
                                     op, ldo, _flat(lse, "lse", "float32", B * n_q),
                                     _stream(stream)))
        return (out, lse) if return_lse else out

    def read(self, slots, dtype=None, k_out=None, v_out=None, stream=None):
        """qmm_kv_read: (k, v) values of the slots, [T, n_kv_heads, head_dim]."""
        import torch
        T, H, D = slots.numel(), self.n_kv_heads, self.head_dim
        dtype = dtype or (k_out.dtype if k_out is not None else torch.float32)
        made = []
        for given in (k_out, v_out):
            if given is None:
                given = torch.empty((T, H, D), dtype=dtype, device=slots.device)
                _made_on(stream, given)
            made.append(given)
        kp, ldk = _heads(made[0], "k_out", T, H, D, dtype)
        vp, ldv = _heads(made[1], "v_out", T, H, D, dtype)
        _check(lib().qmm_kv_read(self.h, _dtype(made[0]), T, _flat(slots, "slots", "int64"), kp,
                                 ldk, vp, ldv, _stream(stream)))
        return made[0], made[1]

    def status(self) -> int:
        """The handle's device status (0 = OK); clears it."""
        return int(lib().qmm_kv_get_status(self.h))


def kv_bytes(kind: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int) -> int:
    """qmm_kv_bytes: the bytes of each of a cache's two buffers."""
    n = int(lib().qmm_kv_bytes(kind, n_pages, page_size, n_kv_heads, head_dim))
    if n < 0:
        _check(n)
    return n


def logits_adjust(logits, out=None, *, history=None, history_offsets=None, repeat=None,
                  presence=None, frequency=None, bias_ids=None, bias_values=None,
                  bias_offsets=None, mask=None, stream=None):
    """qmm_logits_adjust: penalties, biases and a mask on [rows, vocabulary] (or
    one row of) logits.  history, bias_ids: int32, ragged by the rows + 1 int64
    offsets; repeat, presence, frequency: float32 [rows]; mask: int32 words
    [rows, words], or one row [words] for all.  out may be logits."""
    import torch
    if logits.dim() not in (1, 2) or not logits.is_cuda or \
            (logits.shape[-1] > 1 and logits.stride(-1) != 1):
        raise ValueError("logits must be [rows, vocabulary] or [vocabulary] on the CUDA device, "
                         "each row contiguous")
    if out is None:
        out = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        _made_on(stream, out)
    if out.shape != logits.shape or out.dtype != logits.dtype or not out.is_cuda or \
            (out.shape[-1] > 1 and out.stride(-1) != 1):
        raise ValueError("out must be like logits")
    B, V = (1, logits.shape[0]) if logits.dim() == 1 else logits.shape
    ld, ldo = (logits.stride(0), out.stride(0)) if logits.dim() == 2 and B > 1 else (V, V)
    r = LogitRules()
    if history is not None and history.numel():
        r.history = _flat(history, "history", "int32")
        r.history_offsets = _flat(history_offsets, "history_offsets", "int64", B + 1)
        r.n_history = history.numel()
    r.repeat = _flat(repeat, "repeat", "float32", B)
    r.presence = _flat(presence, "presence", "float32", B)
    r.frequency = _flat(frequency, "frequency", "float32", B)
    if bias_ids is not None and bias_ids.numel():
        n = bias_ids.numel()
        r.bias_ids = _flat(bias_ids, "bias_ids", "int32")
        r.bias_values = _flat(bias_values, "bias_values", "float32", n)
        r.bias_offsets = _flat(bias_offsets, "bias_offsets", "int64", B + 1)
        r.n_biases = n
    if mask is not None:
        words = mask.shape[-1]
        if words * 32 < V or mask.numel() not in (words, B * words):
            raise ValueError(f"mask of shape {tuple(mask.shape)} does not hold {B} or 1 rows of "
                             f"{V} bits")
        r.mask = _flat(mask, "mask", "int32")
        r.ld_mask = words if mask.numel() == B * words else 0
    _check(lib().qmm_logits_adjust(_dtype(logits), B, V, logits.data_ptr(), ld, ctypes.byref(r),
                                   out.data_ptr(), ldo, _stream(stream)))
    return out

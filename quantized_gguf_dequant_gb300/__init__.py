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

# These calls are small next to what Python spends on them: checks are plain
# attribute reads, and what they need of torch and of the library is looked up
# once (_ops).
class _Ops:
    """torch, its dtypes, and the C entries, looked up on first use."""

    def __init__(self):
        import torch
        L = lib()
        self.torch, self.empty = torch, torch.empty
        self.f32, self.i32, self.i64 = torch.float32, torch.int32, torch.int64
        self.ids = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
        self.append, self.read, self.attn = L.qmm_kv_append, L.qmm_kv_read, L.qmm_attn_decode
        self.logits = L.qmm_logits_adjust
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

    def type_id(self, dtype) -> int:
        n = self.ids.get(dtype)
        if n is None:
            raise ValueError(f"{dtype} is not supported (float32, float16 and bfloat16 are)")
        return n

    def stream(self, stream, device):
        if stream is None:
            if self.raw_stream is not None:
                return self.raw_stream(device)
            stream = self.torch.cuda.current_stream(device)
        return stream if isinstance(stream, int) else stream.cuda_stream


_the_ops = None


def _ops() -> _Ops:
    global _the_ops
    if _the_ops is None:
        _the_ops = _Ops()
    return _the_ops


def _flat(t, name: str, dtype, n=None):
    """The pointer of a contiguous device tensor of a torch dtype (and, with n
    given, of n elements); None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on the CUDA device")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements; {n} are needed")
    return t.data_ptr()


def _heads(t, name: str, shape, dtype):
    """Elements between the tokens of a [T, heads, D] tensor whose tokens may
    lie apart, such as a slice of a fused projection's output."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; {tuple(shape)} is needed")
    if t.dtype is not dtype:
        raise ValueError(f"{name} is {t.dtype}; {dtype} is needed")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the CUDA device")
    T, heads, D = shape
    a, b, c = t.stride()
    if c != 1 or (b != D and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return a if T > 1 else heads * D


def _made_on(stream, *tensors):
    """Outputs allocated here for work on a stream that is not the current one
    must not return to the allocator before that work is done."""
    if not isinstance(stream, int):
        for t in tensors:
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
                             _flat(inv_freq, "inv_freq", _ops().f32))
        self.ref = ctypes.byref(self.desc)


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
        self._ops, self._device = _ops(), k.device.index or 0
        self._desc = AttnDesc()  # filled anew by each call (a handle serves one stream)
        self._desc_ref = ctypes.byref(self._desc)

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
        o, D, dtype = self._ops, self.head_dim, k.dtype
        T = k.shape[0]
        shape = (T, self.n_kv_heads, D)
        ldk, ldv = _heads(k, "k", shape, dtype), _heads(v, "v", shape, dtype)
        qp = qop = pp = desc = None
        ldq = ldqo = n_q = 0
        if q is not None:
            n_q = q.shape[1]
            shape = (T, n_q, D)
            ldq = _heads(q, "q", shape, dtype)
            if q_out is None:
                q_out = o.empty(shape, dtype=dtype, device=q.device)
                ldqo = n_q * D
                if stream is not None:
                    _made_on(stream, q_out)
            else:
                ldqo = _heads(q_out, "q_out", shape, dtype)
            qp, qop = q.data_ptr(), q_out.data_ptr()
        if rope is not None:
            pp = _flat(pos, "pos", o.i32, rope.n_axes * T)
            desc = rope.ref
        rc = o.append(self.h, o.type_id(dtype), T, k.data_ptr(), ldk, v.data_ptr(), ldv,
                      _flat(slots, "slots", o.i64, T), qp, ldq, n_q, qop, ldqo, pp, desc,
                      o.stream(stream, self._device))
        if rc:
            _check(rc)
        return q_out if q is not None else None

    def attend(self, q, page_table, lens, scale=None, softcap: float = 0.0, window: int = 0,
               alibi=None, out=None, lse=None, return_lse: bool = False, stream=None):
        """qmm_attn_decode: attention of one new token of each sequence.  q:
        [n_seqs, n_q_heads, head_dim]; page_table: [n_seqs, pages] int32; lens:
        [n_seqs] int32; scale: 1/sqrt(head_dim) by default.  Returns out (like
        q), and with return_lse also lse ([n_seqs, n_q_heads] float32)."""
        o = self._ops
        shape, dtype = q.shape, q.dtype
        if len(shape) != 3 or shape[2] != self.head_dim:
            raise ValueError(f"q has shape {tuple(shape)}; [n_seqs, heads, {self.head_dim}] is needed")
        B, n_q, D = shape
        ldq = _heads(q, "q", shape, dtype)
        if out is None:
            out = o.empty(shape, dtype=dtype, device=q.device)
            ldo = n_q * D
            if stream is not None:
                _made_on(stream, out)
        else:
            ldo = _heads(out, "out", shape, dtype)
        lp = None
        if lse is not None:
            lp = _flat(lse, "lse", o.f32, B * n_q)
        elif return_lse:
            lse = o.empty((B, n_q), dtype=o.f32, device=q.device)
            lp = lse.data_ptr()
            if stream is not None:
                _made_on(stream, lse)
        if page_table.dim() != 2 or page_table.shape[0] != B:
            raise ValueError(f"page_table must be [{B}, pages]")
        if page_table.dtype is not o.i32 or not page_table.is_cuda:
            raise ValueError("page_table must be int32 on the CUDA device")
        if not page_table.is_contiguous():  # (the ABI takes a row's length as its stride)
            raise ValueError("page_table must be contiguous")
        d = self._desc
        d.scale = D ** -0.5 if scale is None else scale
        d.softcap, d.window = softcap, window
        d.alibi = None if alibi is None else _flat(alibi, "alibi", o.f32, n_q)
        rc = o.attn(self.h, o.type_id(dtype), B, n_q, q.data_ptr(), ldq, page_table.data_ptr(),
                    page_table.shape[1], _flat(lens, "lens", o.i32, B), self._desc_ref,
                    out.data_ptr(), ldo, lp, o.stream(stream, self._device))
        if rc:
            _check(rc)
        return (out, lse) if return_lse else out

    def read(self, slots, dtype=None, k_out=None, v_out=None, stream=None):
        """qmm_kv_read: (k, v) values of the slots, [T, n_kv_heads, head_dim]."""
        o = self._ops
        T, D = slots.numel(), self.head_dim
        shape = (T, self.n_kv_heads, D)
        dtype = dtype or (k_out.dtype if k_out is not None else o.f32)
        ldk = ldv = self.n_kv_heads * D
        if k_out is None:
            k_out = o.empty(shape, dtype=dtype, device=slots.device)
            if stream is not None:
                _made_on(stream, k_out)
        else:
            ldk = _heads(k_out, "k_out", shape, dtype)
        if v_out is None:
            v_out = o.empty(shape, dtype=dtype, device=slots.device)
            if stream is not None:
                _made_on(stream, v_out)
        else:
            ldv = _heads(v_out, "v_out", shape, dtype)
        rc = o.read(self.h, o.type_id(dtype), T, _flat(slots, "slots", o.i64), k_out.data_ptr(),
                    ldk, v_out.data_ptr(), ldv, o.stream(stream, self._device))
        if rc:
            _check(rc)
        return k_out, v_out

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
    o = _ops()
    shape, dtype, stride = logits.shape, logits.dtype, logits.stride()
    if len(shape) not in (1, 2) or not logits.is_cuda or (stride[-1] != 1 and shape[-1] > 1):
        raise ValueError("logits must be [rows, vocabulary] or [vocabulary] on the CUDA device, "
                         "each row contiguous")
    B, V = shape if len(shape) == 2 else (1, shape[0])
    ld = ldo = V
    if out is None:
        out = o.empty(shape, dtype=dtype, device=logits.device)
        if stream is not None:
            _made_on(stream, out)
    else:
        if out.shape != shape or out.dtype is not dtype or not out.is_cuda or \
                (out.stride(-1) != 1 and V > 1):
            raise ValueError("out must be like logits")
        if B > 1:
            ldo = out.stride(0)
    if B > 1:
        ld = stride[0]
    r = LogitRules()
    f32, i32, i64 = o.f32, o.i32, o.i64
    if history is not None:
        n = history.numel()
        if n:
            r.history = _flat(history, "history", i32)
            r.history_offsets = _flat(history_offsets, "history_offsets", i64, B + 1)
            r.n_history = n
    if repeat is not None:
        r.repeat = _flat(repeat, "repeat", f32, B)
    if presence is not None:
        r.presence = _flat(presence, "presence", f32, B)
    if frequency is not None:
        r.frequency = _flat(frequency, "frequency", f32, B)
    if bias_ids is not None:
        n = bias_ids.numel()
        if n:
            r.bias_ids = _flat(bias_ids, "bias_ids", i32)
            r.bias_values = _flat(bias_values, "bias_values", f32, n)
            r.bias_offsets = _flat(bias_offsets, "bias_offsets", i64, B + 1)
            r.n_biases = n
    if mask is not None:
        words, n = mask.shape[-1], mask.numel()
        if words * 32 < V or (n != words and n != B * words):
            raise ValueError(f"mask of shape {tuple(mask.shape)} does not hold {B} or 1 rows of "
                             f"{V} bits")
        r.mask = _flat(mask, "mask", i32)
        r.ld_mask = words if n == B * words else 0
    rc = o.logits(o.type_id(dtype), B, V, logits.data_ptr(), ld, ctypes.byref(r), out.data_ptr(),
                  ldo, o.stream(stream, logits.device.index))
    if rc:
        _check(rc)
    return out

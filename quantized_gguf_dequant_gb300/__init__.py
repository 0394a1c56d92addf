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

NATIVE_PATH = os.path.join(_HERE, "_native.so")
_native = None


def native():
    """The module behind the calls below (csrc/binding.cpp): it takes tensors
    apart, checks them and calls the C ABI of the loaded library."""
    global _native
    if _native is None:
        import importlib.machinery
        import importlib.util

        import torch  # noqa: F401  (its libraries must be loaded first)
        L = lib()
        if not os.path.exists(NATIVE_PATH):
            raise RuntimeError(
                f"{NATIVE_PATH} is missing: build it with "
                "`python -m quantized_gguf_dequant_gb300.build` (there is no fallback)")
        loader = importlib.machinery.ExtensionFileLoader("_native", NATIVE_PATH)
        spec = importlib.util.spec_from_file_location("_native", NATIVE_PATH, loader=loader)
        m = importlib.util.module_from_spec(spec)
        loader.exec_module(m)
        m.init(QmmError, *(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in (
            "qmm_kv_append", "qmm_kv_read", "qmm_attn_decode", "qmm_logits_adjust",
            "qmm_last_error")))
        _native = m
    return _native


class Rope:
    """Rotary positions: inv_freq (fp32 on the device, one per pair), the pairs
    that turn by each axis (sections; default: one axis), and which dims are
    a pair: "halves" (i, i + n_rot/2) or "adjacent" (2i, 2i + 1)."""

    def __init__(self, inv_freq, sections=None, pairing: str = "halves"):
        import torch
        n = inv_freq.numel()
        sections = [n] if sections is None else [int(x) for x in sections]
        if pairing not in ("halves", "adjacent"):
            raise ValueError(f"pairing {pairing!r}: 'halves' or 'adjacent'")
        if not 1 <= len(sections) <= 4 or sum(sections) != n:
            raise ValueError(f"sections {sections} must be 1 to 4 counts that sum to {n} pairs")
        if inv_freq.dtype != torch.float32 or not inv_freq.is_cuda or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float32 tensor on the CUDA device")
        self.inv_freq = inv_freq  # keep the device memory alive
        self.device = inv_freq.device.index
        self.desc = RopeDesc(2 * n, int(pairing == "adjacent"), len(sections),
                             (ctypes.c_int32 * 4)(*sections), inv_freq.data_ptr())
        self.address = ctypes.addressof(self.desc)


class KVCache:
    """A paged key-value cache on the device (qmm_kv_create) with the calls
    that use it.  kind: F16, BF16 or Q8_0.  k, v: its two buffers (any dtype,
    at least kv_bytes() bytes each, on the current device); made and zeroed here
    when not given.  Every call takes a stream (a torch stream or a raw handle;
    default: the current one).  Calls on one cache share its workspace and must
    be ordered, as on one stream.  On another stream than the current one a call waits for
    nothing: its inputs must be ready there (stream.wait_stream), but may be
    dropped at once."""

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
            # the handle belongs to the current device, and so do its calls
            if not t.is_cuda or t.device.index != torch.cuda.current_device():
                raise ValueError(f"the {name} buffer lives on {t.device}, but device "
                                 f"{torch.cuda.current_device()} is current")
        self.k, self.v = k, v  # keep the buffers alive as long as the handle
        self._native = native()
        h = ctypes.c_void_p()
        _check(lib().qmm_kv_create(kind, n_pages, page_size, n_kv_heads, head_dim, _ptr(k),
                                   _ptr(v), ctypes.byref(h)))
        self.h = h.value
        self._cache = self._native.cache(self.h, k.device.index, n_kv_heads, head_dim)

    def close(self):
        if getattr(self, "h", None):
            h, self.h, self._cache = self.h, None, None
            _check(lib().qmm_kv_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def append(self, k, v, slots, q=None, pos=None, rope=None, q_out=None, stream=None):
        """qmm_kv_append: rotate q and k ([T, heads, head_dim]) and store k and
        v at slots ([T] int64).  pos: [n_axes, T] int32 (one axis: [T] will do).  Returns the
        rotated q (into q_out, which may be q), or None without q."""
        return self._native.append(self._cache, k, v, slots, q, pos, rope, q_out, stream)

    def attend(self, q, page_table, lens, scale=None, softcap: float = 0.0, window: int = 0,
               alibi=None, out=None, lse=None, return_lse: bool = False, stream=None):
        """qmm_attn_decode: attention of one new token of each sequence.  q:
        [n_seqs, n_q_heads, head_dim]; page_table: [n_seqs, pages] int32; lens:
        [n_seqs] int32; scale: 1/sqrt(head_dim) by default.  Returns out (like
        q), and with return_lse also lse ([n_seqs, n_q_heads] float32)."""
        return self._native.attend(self._cache, q, page_table, lens, scale, softcap, window, alibi,
                                   out, lse, return_lse, stream)

    def read(self, slots, dtype=None, k_out=None, v_out=None, stream=None):
        """qmm_kv_read: (k, v) values of the slots, [T, n_kv_heads, head_dim], in
        dtype (default: that of the output that is given, else float32)."""
        return self._native.read(self._cache, slots, dtype, k_out, v_out, stream)

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
    one row of) logits on the current device.  history, bias_ids: int32, ragged by the rows + 1 int64
    offsets; repeat, presence, frequency: float32 [rows]; mask: int32 words
    [rows, words], or one row [words] for all.  out may be logits.  stream: as
    for a KVCache's calls."""
    return (_native or native()).logits(logits, out, history, history_offsets, repeat, presence,
                                        frequency, bias_ids, bias_values, bias_offsets, mask,
                                        stream)

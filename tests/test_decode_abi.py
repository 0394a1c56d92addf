"""The decode-step operators without a GPU: what the host refuses by name
before it touches the device, and the cache's sizes."""
from __future__ import annotations

import ctypes

import pytest

import quantized_gguf_dequant_gb300 as q
from quantized_gguf_dequant_gb300 import build as qbuild


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return q.lib()


def create(kind=q.F16, pages=4, page=16, heads=2, D=64, k=0x10000, v=0x20000):
    h = ctypes.c_void_p()
    rc = q.lib().qmm_kv_create(kind, pages, page, heads, D, ctypes.c_void_p(k), ctypes.c_void_p(v),
                               ctypes.byref(h))
    assert h.value is None
    return rc, q.last_error()


def test_create_refuses_by_name(L):
    rc, msg = create(kind=12)
    assert rc == q.ERR_FORMAT and "type 12" in msg
    for bad in (dict(pages=0), dict(page=0), dict(heads=0), dict(pages=-1)):
        assert create(**bad)[0] == q.ERR_SHAPE
    rc, msg = create(D=80)
    assert rc == q.ERR_UNSUPPORTED and "head_dim = 80" in msg
    assert create(pages=1 << 40)[0] == q.ERR_SHAPE
    assert create(pages=2, page=2 ** 31 - 1, heads=2)[0] == q.ERR_SHAPE
    rc, msg = create(v=0)
    assert rc == q.ERR_NULL and "value" in msg
    rc, msg = create(k=0x10008)
    assert rc == q.ERR_ALIGN and "key" in msg
    assert L.qmm_kv_create(q.F16, 4, 16, 2, 64, ctypes.c_void_p(16), ctypes.c_void_p(16),
                           None) == q.ERR_NULL


@pytest.mark.parametrize("kind,D,row", [(q.F16, 64, 128), (q.BF16, 96, 192), (q.Q8_0, 64, 68),
                                        (q.Q8_0, 96, 104), (q.Q8_0, 128, 136), (q.Q8_0, 192, 204),
                                        (q.Q8_0, 256, 272)])
def test_sizes(L, kind, D, row):
    assert q.kv_bytes(kind, 5, 7, 3, D) == 5 * 7 * 3 * row
    with pytest.raises(q.QmmError):
        q.kv_bytes(kind, 5, 7, 3, D + 1)


def test_more_heads_than_fit_refuse():
    assert q.kv_bytes(q.F16, 1, 1, 1 << 20, 64) == (1 << 20) * 128
    with pytest.raises(q.QmmError, match="n_kv_heads"):
        q.kv_bytes(q.F16, 1, 1, (1 << 20) + 1, 64)


def test_null_handles_refuse(L):
    vp = ctypes.c_void_p
    assert L.qmm_kv_append(None, 0, 1, vp(16), 64, vp(16), 64, vp(16), None, 0, 0, None, 0, None,
                           None, None) == q.ERR_NULL
    assert "handle is NULL" in q.last_error()
    assert L.qmm_kv_read(None, 0, 1, vp(16), vp(16), 64, None, 0, None) == q.ERR_NULL
    d = q.AttnDesc(1.0, 0.0, 0, None)
    assert L.qmm_attn_decode(None, 0, 1, 1, vp(16), 64, vp(16), 1, vp(16), ctypes.byref(d), vp(16),
                             64, None, None) == q.ERR_NULL
    assert L.qmm_kv_get_status(None) == q.ERR_NULL and L.qmm_kv_destroy(None) == q.ERR_NULL


def test_type_ids_are_ggufs():
    assert (q.F32, q.F16, q.BF16) == (0, 1, 30)

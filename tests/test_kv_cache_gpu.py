"""New tokens into the paged cache and values out of it (qmm_kv_append,
qmm_kv_read): rotary positions with one to four axes against a 64-bit
restatement, the stored bits against the formats' definitions, slots that are
not to be written, strides, in-place queries, and refusals."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from tests import _decode_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")

KIND = {"f16": q.F16, "bf16": q.BF16, "q8_0": q.Q8_0}


def quantize(x):
    """Q8_0 by its definition in fp32: (codes, fp16 scales)."""
    b = x.astype(np.float32).reshape(x.shape[:-1] + (-1, 32))
    d = np.abs(b).max(-1) / np.float32(127)
    inv = np.divide(np.float32(1), d, out=np.zeros_like(d), where=d > 0)
    return np.rint(b * inv[..., None]).astype(np.int8).reshape(x.shape), d.astype(np.float16)


def stored(cache, page, heads, D, kind):
    """The two buffers' contents as values [slots, heads, D] (fp64), and as raw arrays."""
    out = []
    for buf in (cache.k, cache.v):
        raw = buf.view(torch.uint8).reshape(-1).cpu()
        n = cache.n_pages * heads * page * D
        if kind == "q8_0":
            codes = raw[:n].view(torch.int8).numpy().reshape(-1, heads, page, D)
            scales = raw[n:].view(torch.float16).numpy().reshape(codes.shape[:3] + (-1,))
            val = codes.astype(np.float64) * np.repeat(
                scales[..., :D // 32].astype(np.float64), 32, axis=-1)
            out.append((val.transpose(0, 2, 1, 3).reshape(-1, heads, D),
                        codes.transpose(0, 2, 1, 3).reshape(-1, heads, D),
                        scales.transpose(0, 2, 1, 3).reshape(-1, heads, scales.shape[-1])))
        else:
            val = raw.view(ref.TORCH_IO[kind]).double().numpy().reshape(-1, heads, page, D)
            out.append((val.transpose(0, 2, 1, 3).reshape(-1, heads, D),))
    return out


def run(kind, T, heads, group, D, page, io="f32", n_rot=None, sections=None, pairing="halves",
        seed=0, in_place=False, top=5000):
    rng = np.random.default_rng(seed)
    nq = heads * group
    n_pages = -(-T // page) + 3
    cache = q.KVCache(KIND[kind], n_pages, page, heads, D)
    for b in (cache.k, cache.v):
        b.fill_(0x3A)
    before = stored(cache, page, heads, D, kind)
    qkv = torch.from_numpy(rng.standard_normal((T, nq + 2 * heads, D)).astype(np.float32))
    qkv = qkv.to(ref.TORCH_IO[io]).cuda()
    xq, xk, xv = qkv.split([nq, heads, heads], dim=1)
    host = [t.double().cpu().numpy() for t in (xq, xk, xv)]
    slots = rng.permutation(n_pages * page)[:T].astype(np.int64)
    if T >= 3:
        slots[T // 2] = -1
    n_rot = D if n_rot is None else n_rot
    half = n_rot // 2
    sections = [half] if sections is None else sections
    pos = rng.integers(0, top, (len(sections), T)).astype(np.int32)
    inv = (10000.0 ** (-np.arange(half) / max(1, half))).astype(np.float32)
    rope = q.Rope(torch.from_numpy(inv).cuda(), sections, pairing) if half else None
    got = cache.append(xk, xv, torch.from_numpy(slots).cuda(), q=xq,
                       pos=torch.from_numpy(pos).cuda(), rope=rope,
                       q_out=xq if in_place else None)
    assert cache.status() == q.OK, q.last_error()
    assert got.shape == (T, nq, D) and got.dtype == qkv.dtype
    wq, wk = (ref.rotate(x, pos, inv, sections, pairing) if half else x for x in host[:2])
    tq, tk = (ref.rotation_bound(x, n_rot, pairing) for x in host[:2])
    err = np.abs(got.double().cpu().numpy() - wq)
    tiny = 2.0 ** -24 if io == "f16" else 0
    assert (err <= tq * (1 + ref.ROUND[io]) + np.abs(wq) * ref.ROUND[io] + tiny).all()
    after = stored(cache, page, heads, D, kind)
    kept = slots >= 0
    untouched = np.ones(n_pages * page, bool)
    untouched[slots[kept]] = False
    for a, b in zip(after, before):
        for x, y in zip(a, b):
            assert np.array_equal(x[untouched], y[untouched], equal_nan=True)
    sel = slots[kept]
    if kind == "q8_0":
        # values are not rotated: their codes and scales are exactly the definition's
        codes, scales = quantize(host[2])
        assert np.array_equal(after[1][1][sel], codes[kept])
        assert np.array_equal(after[1][2][sel][..., :D // 32], scales[kept])
        d = np.abs(wk.reshape(T, heads, -1, 32)).max(-1) / 127
        d = np.repeat(d, 32, axis=-1)[kept]
        # half a code, what the scale's own rounding moves, and the rotation's error
        bound = d * (0.5 + 127 * 2.0 ** -11 + 2.0 ** -12) + 130 / 127 * tk[kept].max(-1, keepdims=True)
        assert (np.abs(after[0][0][sel] - wk[kept]) <= bound).all()
    else:
        r = ref.ROUND[kind]
        v32 = torch.from_numpy(host[2].astype(np.float32)).to(ref.TORCH_IO[kind]).double().numpy()
        assert np.array_equal(after[1][0][sel], v32[kept])
        tol = tk * (1 + r) + np.abs(wk) * r + (2.0 ** -24 if kind == "f16" else 0)
        assert (np.abs(after[0][0][sel] - wk[kept]) <= tol[kept]).all()
    cache.close()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("T", [1, 2, 37])
def test_append(kind, D, T):
    run(kind, T, 2, 3, D, 16, seed=D + T)


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
@pytest.mark.parametrize("D,n_rot,sections", [
    (128, 128, [16, 24, 24]), (128, 64, [8, 0, 24]), (96, 96, [1, 2, 3, 42]), (64, 2, [1]),
    (64, 6, [1, 2]), (64, 0, None), (96, 24, [12]), (256, 250, [100, 25]), (192, 190, [95]),
])
def test_axes_and_partial_rotation(kind, pairing, D, n_rot, sections):
    run(kind, 9, 2, 2, D, 5, n_rot=n_rot, sections=sections, pairing=pairing, seed=n_rot)


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
def test_types(io, kind):
    run(kind, 21, 3, 2, 128, 7, io=io)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 256])
@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
def test_queries_rotated_in_place(io, D, pairing):
    run("bf16", 40, 2, 4, D, 16, io=io, pairing=pairing, in_place=True)


@pytest.mark.parametrize("kind", ["f16", "q8_0"])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,n_rot", [(64, 32), (96, 96), (96, 36), (128, 64), (128, 100), (192, 96),
                                     (192, 184), (256, 64), (256, 254)])
@pytest.mark.parametrize("heads,group,in_place", [(1, 1, True), (3, 5, True), (2, 8, False)])
def test_partial_rotation_of_every_type(kind, io, D, n_rot, heads, group, in_place):
    run(kind, 12, heads, group, D, 16, io=io, n_rot=n_rot, in_place=in_place, seed=D + n_rot)


@pytest.mark.parametrize("n_rot,pairing", [(64, "halves"), (24, "halves"), (20, "adjacent")])
def test_whole_tokens_of_partial_rotation(n_rot, pairing):
    run("q8_0", 700, 3, 7, 96, 16, io="bf16", n_rot=n_rot, pairing=pairing, in_place=True)


def test_large_positions():
    run("bf16", 30, 1, 2, 64, 16, top=2 ** 31 - 1, seed=3)
    run("bf16", 30, 1, 2, 64, 16, top=200000, seed=4)


@pytest.mark.parametrize("heads,group,D", [(1, 1, 64), (8, 4, 128), (3, 71, 64)])
@pytest.mark.parametrize("T", [1, 700])
def test_head_counts(heads, group, D, T):
    run("f16", T, heads, group, D, 16, seed=heads)


def test_without_queries_or_rotation():
    cache = q.KVCache(q.F16, 2, 16, 2, 64)
    x = torch.randn(3, 2, 64, device="cuda")
    slots = torch.tensor([0, 31, 5], device="cuda")
    assert cache.append(x, 2 * x, slots) is None
    k, v = cache.read(slots)
    assert torch.equal(k, x.half().float()) and torch.equal(v, (2 * x).half().float())
    assert cache.append(x[:0], x[:0], slots[:0]) is None  # no tokens: nothing to do
    assert cache.status() == q.OK


def test_slots_outside_the_cache():
    cache = q.KVCache(q.Q8_0, 2, 16, 2, 64)
    cache.k.fill_(1)
    keep = cache.k.clone()
    x = torch.randn(3, 2, 64, device="cuda")
    xq = torch.randn(3, 2, 64, device="cuda")
    slots = torch.tensor([32, -7, 2 ** 62], device="cuda")
    got = cache.append(x, x, slots, q=xq)
    assert torch.equal(got, xq) and torch.equal(cache.k, keep)
    assert cache.status() == q.ERR_PAGE and "slot" in q.last_error()
    k, v = cache.read(slots)
    assert (k == 0).all() and (v == 0).all()
    assert cache.status() == q.ERR_PAGE
    assert cache.status() == q.OK
    cache.append(x, x, torch.full((3,), -1, device="cuda"))
    assert cache.status() == q.OK  # padding is no fault


def test_q8_special_blocks():
    """Zero blocks, ties to even, tiny and huge values, infinities and NaN."""
    x = np.zeros((6, 1, 64), np.float32)
    x[1, 0, :5] = [-127.0, 0.5, 1.5, 2.5, -0.5]
    x[2, 0] = np.linspace(-1e-30, 1e-30, 64)
    x[3, 0] = np.linspace(-1e6, 1e6, 64)
    x[4, 0, 3], x[4, 0, 40] = np.inf, 1.0
    x[5, 0, 3], x[5, 0, 40] = np.nan, 1.0
    cache = q.KVCache(q.Q8_0, 1, 8, 1, 64)
    t = torch.from_numpy(x).cuda()
    slots = torch.arange(6, device="cuda")
    cache.append(t, t, slots)
    codes, scales = quantize(x[:4])
    (_, gc, gs), _ = stored(cache, 8, 1, 64, "q8_0")
    assert np.array_equal(gc[:4], codes) and np.array_equal(gs[:4], scales)
    k, _ = cache.read(slots)
    k = k.cpu().numpy()
    assert not np.isfinite(k[4, 0, 3]) and np.isnan(k[5, 0, 3])  # the fault shows
    assert k[4, 0, 40] == k[5, 0, 40] == np.float32(127) * np.float32(np.float16(np.float32(1) / 127))


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 96, 256])
def test_read(kind, io, D):
    rng = np.random.default_rng(D)
    pages = ref.Pages(q, kind, 5, 13, 3, D, rng)
    cache = pages.to_device(np.arange(65))
    slots = rng.integers(0, 65, 50).astype(np.int64)
    slots[7] = -1
    dt = ref.TORCH_IO[io]
    out = torch.full((50, 8, D), 3.0, dtype=dt, device="cuda")
    k, v = cache.read(torch.from_numpy(slots).cuda(), k_out=out[:, 1:4], v_out=out[:, 5:8])
    assert (out[:, 0] == 3).all() and (out[:, 4] == 3).all()
    for got, which in ((k, 0), (v, 1)):
        want = torch.from_numpy(pages.rows(which, np.maximum(slots, 0)).astype(np.float32)).to(dt)
        want[7] = 0
        assert torch.equal(got.cpu(), want)
    assert cache.read(torch.from_numpy(slots[:0]).cuda())[0].shape == (0, 3, D)


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_on_another_stream(raw):
    # what a call on another stream returns is that stream's memory: the
    # current stream's next tensors cannot take its place while it is written
    rng = np.random.default_rng(4)
    cache = q.KVCache(q.F16, 20, 16, 2, 64)
    x = torch.from_numpy(rng.standard_normal((300, 2, 64)).astype(np.float16)).cuda()
    slots = torch.arange(300, device="cuda")
    cache.append(x, x, slots)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on = s.cuda_stream if raw else s
    k, v = cache.read(slots, torch.float16, stream=on)
    turned = cache.append(x, x, slots, q=x, stream=on)
    y = q.logits_adjust(x.view(300, 128), stream=on)
    s.synchronize()
    assert torch.equal(k, x) and torch.equal(v, x)
    assert torch.equal(turned, x) and torch.equal(y, x.view(300, 128))
    torch.cuda.synchronize()
    taken = {t.data_ptr() for t in (k, v, turned, y)}
    del k, v, turned, y
    new = [torch.empty((300, 2, 64), dtype=torch.float16, device="cuda") for _ in range(8)]
    assert not taken & {t.data_ptr() for t in new}
    cache.close()


def test_refusals():
    cache = q.KVCache(q.F16, 2, 16, 2, 64)
    x = torch.randn(3, 2, 64, device="cuda")
    slots = torch.tensor([0, 1, 2], device="cuda")
    L, vp, p = q.lib(), ctypes.c_void_p, x.data_ptr()
    inv = torch.ones(32, device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    good = q.RopeDesc(64, 0, 1, (ctypes.c_int32 * 4)(32), inv.data_ptr())

    def call(dtype=q.F32, T=3, k=p, ldk=128, s=slots.data_ptr(), qp=p, ldq=128, nq=2, qo=p,
             ldqo=128, pp=pos.data_ptr(), rope=good):
        before = q.launch_count()
        rc = L.qmm_kv_append(cache.h, dtype, T, vp(k), ldk, vp(p), 128, vp(s), vp(qp), ldq, nq,
                             vp(qo), ldqo, vp(pp), ctypes.byref(rope), None)
        assert q.launch_count() == before
        return rc

    assert call(dtype=30000) == q.ERR_FORMAT and call(T=-1) == q.ERR_SHAPE
    assert call(k=0) == q.ERR_NULL and "k is NULL" in q.last_error()
    assert call(s=0) == q.ERR_NULL and call(qo=0) == q.ERR_NULL and call(pp=0) == q.ERR_NULL
    assert call(k=p + 8) == q.ERR_ALIGN and call(ldk=130) == q.ERR_ALIGN
    assert call(ldk=64) == q.ERR_SHAPE and call(nq=0) == q.ERR_SHAPE
    assert call(ldqo=256) == q.ERR_SHAPE and "q_out is q" in q.last_error()
    for rope, code in ((q.RopeDesc(63, 0, 1, (ctypes.c_int32 * 4)(31), inv.data_ptr()), q.ERR_SHAPE),
                       (q.RopeDesc(66, 0, 1, (ctypes.c_int32 * 4)(33), inv.data_ptr()), q.ERR_SHAPE),
                       (q.RopeDesc(64, 2, 1, (ctypes.c_int32 * 4)(32), inv.data_ptr()),
                        q.ERR_UNSUPPORTED),
                       (q.RopeDesc(64, 0, 5, (ctypes.c_int32 * 4)(32), inv.data_ptr()), q.ERR_SHAPE),
                       (q.RopeDesc(64, 0, 2, (ctypes.c_int32 * 4)(33, -1), inv.data_ptr()),
                        q.ERR_SHAPE),
                       (q.RopeDesc(64, 0, 2, (ctypes.c_int32 * 4)(16, 15), inv.data_ptr()),
                        q.ERR_SHAPE),
                       (q.RopeDesc(64, 0, 1, (ctypes.c_int32 * 4)(32), None), q.ERR_NULL)):
        assert call(rope=rope) == code
    before = q.launch_count()
    assert L.qmm_kv_read(cache.h, q.F32, 3, vp(slots.data_ptr()), None, 0, None, 0,
                         None) == q.ERR_NULL
    assert L.qmm_kv_read(cache.h, q.F32, 3, None, vp(p), 128, None, 0, None) == q.ERR_NULL
    assert L.qmm_kv_read(cache.h, q.F32, 3, vp(slots.data_ptr()), vp(p), 126, None, 0,
                         None) == q.ERR_SHAPE
    assert q.launch_count() == before
    for bad in (dict(k=x.double()), dict(k=x[:, :1]), dict(slots=slots.int()),
                dict(v=x[..., ::2]), dict(slots=slots[:2])):
        a = dict(k=x, v=x, slots=slots)
        a.update(bad)
        with pytest.raises(ValueError):
            cache.append(**a)
    with pytest.raises(ValueError):
        q.KVCache(q.F16, 2, 16, 2, 64, k=torch.zeros(10, device="cuda"))

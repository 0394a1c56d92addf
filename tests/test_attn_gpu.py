"""Attention of one new token over the paged cache (qmm_attn_decode) against a
64-bit restatement: every cache type and head size, lengths around the tile
and block borders, pages that end inside a tile, caps, biases and windows,
stale NaNs in every slot that is not in range, and what a call must refuse."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

from tests import _decode_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")

KINDS = ["f16", "bf16", "q8_0"]


def check(kind, lens, heads, group, D, page, io="f32", seed=0, scale=None, softcap=0.0, window=0,
          alibi=False, strided=False):
    rng = np.random.default_rng(seed)
    B, nq = len(lens), heads * group
    table, n_pages, slots = ref.table_for(lens, page, rng)
    pages = ref.Pages(q, kind, n_pages, page, heads, D, rng)
    used = [s[max(0, len(s) - window) if window else 0:] for s in slots]
    cache = pages.to_device(np.concatenate(used))
    scale = 1 / math.sqrt(D) if scale is None else scale
    x = torch.from_numpy(rng.standard_normal((B, nq + 3, D)).astype(np.float32)).to(ref.TORCH_IO[io])
    x = x.cuda()
    x = x[:, 1:1 + nq] if strided else x[:, :nq].contiguous()
    slope = (2.0 ** -(8 * (np.arange(nq) + 1) / nq)).astype(np.float32) if alibi else None
    out = torch.full((B, nq + 5, D), 7.0, dtype=x.dtype, device="cuda")
    view = out[:, 2:2 + nq]
    got, lse = cache.attend(x, torch.from_numpy(table).cuda(),
                            torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=scale,
                            softcap=softcap, window=window, out=view if strided else None,
                            alibi=torch.from_numpy(slope).cuda() if alibi else None,
                            return_lse=True)
    assert cache.status() == q.OK, q.last_error()
    if strided:  # nothing beside the rows was written
        assert (out[:, :2] == 7).all() and (out[:, 2 + nq:] == 7).all()
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    x = x.double().cpu().numpy()
    scale32 = float(np.float32(scale))
    for b in range(B):
        want, want_lse, size = ref.attention(x[b], pages.rows(0, slots[b]), pages.rows(1, slots[b]),
                                             scale32, softcap, window,
                                             None if slope is None else slope.astype(np.float64))
        tol, tol_lse = ref.attention_bound(size, D)
        tol = tol[:, None] + np.abs(want) * 1.01 * ref.ROUND[io] + (1e-7 if io == "f16" else 0)
        err = np.abs(got[b] - want)
        assert np.isfinite(got[b]).all(), (b, lens[b])
        assert (err <= tol).all(), (b, lens[b], float((err / np.maximum(tol, 1e-300)).max()))
        if lens[b] == 0:
            assert (got[b] == 0).all() and (lse[b] == -np.inf).all()
        else:
            assert (np.abs(lse[b] - want_lse) <= tol_lse).all(), (b, lens[b])
    cache.close()


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 200]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("group,page", [(1, 16), (4, 24), (8, 5)])
def test_lengths(kind, D, group, page):
    check(kind, LENS, 2, group, D, page, seed=D + group)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group", [2, 3, 5, 7, 9, 12, 16, 17])
def test_groups(kind, group):
    check(kind, [33, 0, 70], 3, group, 64, 16, seed=group)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 2, 7, 16, 17, 64, 100, 1000])
def test_pages_that_end_inside_a_tile(kind, page):
    check(kind, [1, 100, 257], 2, 4, 128, page, seed=page)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("io", ["f32", "f16", "bf16"])
def test_types_and_strides(kind, io):
    check(kind, [5, 40, 300], 2, 4, 128, 16, io=io, strided=True, seed=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 5, 16, 31, 64, 10000])
def test_windows(kind, window):
    check(kind, [0, 1, 4, 16, 40, 129], 2, 2, 64, 24, window=window, seed=window)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("softcap,alibi,window", [(30.0, False, 0), (0.0, True, 0), (2.0, True, 50),
                                                  (50.0, True, 0)])
def test_caps_and_biases(kind, softcap, alibi, window):
    check(kind, [1, 77, 400], 2, 6, 128, 16, softcap=softcap, alibi=alibi, window=window,
          scale=0.4, seed=11)


@pytest.mark.parametrize("kind,D", [("bf16", 128), ("f16", 64), ("q8_0", 128), ("q8_0", 96),
                                    ("f16", 256)])
def test_one_long_sequence_joined_from_many_blocks(kind, D):
    check(kind, [9001], 2, 4, D, 32, seed=5)


@pytest.mark.parametrize("kind", KINDS)
def test_more_sequences_than_threads(kind):
    rng = np.random.default_rng(8)
    lens = [int(n) for n in rng.integers(0, 60, 300)]
    lens[0] = lens[299] = 0
    lens[150] = 700
    check(kind, lens, 2, 2, 64, 16, seed=9)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,longest", [(32, 900), (33, 40), (33, 2500), (64, 700), (97, 60),
                                       (128, 30), (128, 1500), (129, 300)])
def test_counts_of_sequences(kind, B, longest):
    rng = np.random.default_rng(B + longest)
    lens = [int(n) for n in rng.integers(0, 40, B)]
    lens[0] = lens[B // 2] = 0
    lens[B - 1] = lens[B // 3] = longest
    check(kind, lens, 1, 4, 64, 16, seed=B)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,group,page", [(128, 4, 16), (128, 8, 16), (128, 3, 24), (128, 16, 16),
                                          (256, 4, 16), (96, 7, 16)])
def test_batches_of_wide_rows(kind, D, group, page):
    rng = np.random.default_rng(D + group)
    lens = [int(n) for n in rng.integers(0, 120, 24)]
    lens[3], lens[11], lens[23] = 1900, 0, 1025
    check(kind, lens, 3, group, D, page, seed=D)


def test_many_sequences_all_empty_but_the_last():
    check("f16", [0] * 99 + [17], 2, 2, 64, 16)
    check("f16", [0] * 77, 2, 2, 64, 16)


def test_lengths_outside_the_table_are_cut_among_many():
    rng = np.random.default_rng(21)
    lens = [16] * 70
    table, n_pages, slots = ref.table_for(lens, 16, rng)
    pages = ref.Pages(q, "f16", n_pages, 16, 1, 64, rng)
    cache = pages.to_device(np.concatenate(slots))
    x = torch.from_numpy(rng.standard_normal((70, 2, 64)).astype(np.float32)).cuda()
    run = lambda n: cache.attend(x, torch.from_numpy(table).cuda(), torch.tensor(
        n, dtype=torch.int32, device="cuda"), scale=0.125)
    want = run(lens)
    assert cache.status() == q.OK
    lens[41] = 1000  # past the table: as its 16 slots
    got = run(lens)
    assert torch.equal(got, want)
    assert cache.status() != q.OK
    lens[41], lens[69] = 16, -5  # below zero: empty
    got = run(lens)
    assert torch.equal(got[:69], want[:69]) and (got[69] == 0).all()
    assert cache.status() != q.OK
    cache.close()


def test_all_sequences_empty():
    check("bf16", [0, 0, 0], 2, 2, 64, 16)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [1e-3, -0.3, 4.0])
def test_flat_and_sharp_scores(kind, scale):
    check(kind, [3, 90, 500], 1, 4, 64, 16, scale=scale, seed=13)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1e-20, 1e-6, 1e6, 1e20])
def test_queries_of_any_size(kind, size):
    """The pieces of q follow its magnitude: scores with scale = 1/size are those of size 1."""
    rng = np.random.default_rng(21)
    table, n_pages, slots = ref.table_for([150], 16, rng)
    pages = ref.Pages(q, kind, n_pages, 16, 2, 64, rng)
    cache = pages.to_device(slots[0])
    x = rng.standard_normal((1, 4, 64)).astype(np.float32)
    big = (x * np.float32(size)).astype(np.float32)
    scale = float(np.float32(0.125 / size))
    out = cache.attend(torch.from_numpy(big).cuda(), torch.from_numpy(table).cuda(),
                       torch.tensor([150], dtype=torch.int32, device="cuda"), scale=scale)
    want, _, bound = ref.attention(big[0].astype(np.float64), pages.rows(0, slots[0]),
                                   pages.rows(1, slots[0]), scale)
    tol, _ = ref.attention_bound(bound, 64)
    assert (np.abs(out[0].double().cpu().numpy() - want) <= tol[:, None]).all()


@pytest.mark.parametrize("size", [1e-4, 1.0, 1000.0])
def test_q8_value_scales_of_mixed_sizes(size):
    """Value scales that differ by orders of magnitude between keys and blocks."""
    rng = np.random.default_rng(31)
    table, n_pages, slots = ref.table_for([400], 16, rng)
    pages = ref.Pages(q, "q8_0", n_pages, 16, 1, 64, rng)
    scales = pages.raw[1][1]
    shape = scales[..., :2].shape
    scales[..., :2] = (size * 10.0 ** rng.uniform(-3, 0, shape)).astype(np.float16)
    scales[..., :2] *= np.where(rng.random(shape) < 0.5, -1, 1)
    pages.val[1] = pages.raw[1][0].astype(np.float64) * np.repeat(
        scales[..., :2].astype(np.float64), 32, axis=-1)
    cache = pages.to_device(slots[0])
    x = rng.standard_normal((1, 2, 64)).astype(np.float32)
    out = cache.attend(torch.from_numpy(x).cuda(), torch.from_numpy(table).cuda(),
                       torch.tensor([400], dtype=torch.int32, device="cuda"))
    want, _, bound = ref.attention(x[0].astype(np.float64), pages.rows(0, slots[0]),
                                   pages.rows(1, slots[0]), 0.125)
    tol, _ = ref.attention_bound(bound, 64)
    assert (np.abs(out[0].double().cpu().numpy() - want) <= tol[:, None]).all()


def _small(kind="f16", n=40, seed=1, D=64):
    rng = np.random.default_rng(seed)
    table, n_pages, slots = ref.table_for([n], 16, rng)
    pages = ref.Pages(q, kind, n_pages, 16, 2, D, rng)
    x = torch.from_numpy(rng.standard_normal((1, 4, D)).astype(np.float32)).cuda()
    return pages, table, slots[0], x, torch.tensor([n], dtype=torch.int32, device="cuda")


def test_infinite_and_nan_values_in_range():
    for kind in ("f16", "bf16"):
        pages, table, slots, x, lens = _small(kind)
        raw = pages.raw[1][0]
        raw[slots[7] // 16, 0, slots[7] % 16, 3] = math.nan    # a value of kv head 0
        raw[slots[9] // 16, 1, slots[9] % 16, 5] = math.inf    # and of kv head 1
        out = pages.to_device(slots).attend(x, torch.from_numpy(table).cuda(), lens).cpu()
        bad = torch.zeros(4, 64, dtype=torch.bool)
        bad[:2, 3] = True
        assert torch.equal(torch.isnan(out[0]), bad)
        assert (out[0, 2:, 5] == math.inf).all()
        assert torch.isfinite(out[0][~bad]).sum() == bad.numel() - 2 - 2
        # a key of -inf against a positive query component is never attended to
        pages, table, slots, x, lens = _small(kind)
        raw = pages.raw[0][0]
        raw[slots[3] // 16, :, slots[3] % 16] = 0
        raw[slots[3] // 16, :, slots[3] % 16, 0] = -math.inf
        x[..., 0] = x[..., 0].abs()
        out = pages.to_device(slots).attend(x, torch.from_numpy(table).cuda(), lens)
        k, v = pages.rows(0, slots), pages.rows(1, slots)
        keep = np.arange(40) != 3
        want, _, size = ref.attention(x[0].double().cpu().numpy(), k[keep], v[keep], 0.125)
        tol, _ = ref.attention_bound(size, 64)
        assert (np.abs(out[0].double().cpu().numpy() - want) <= tol[:, None]).all()


def test_nan_query_stays_in_its_head():
    for kind in KINDS:
        pages, table, slots, x, lens = _small(kind)
        x[0, 1, 5] = math.nan
        x[0, 2, 5] = math.inf
        out = pages.to_device(slots).attend(x, torch.from_numpy(table).cuda(), lens).cpu()
        assert torch.isnan(out[0, 1]).all() and torch.isnan(out[0, 2]).all()
        assert torch.isfinite(out[0, 0]).all() and torch.isfinite(out[0, 3]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_pages_outside_the_cache_are_left_out(kind):
    pages, table, slots, x, lens = _small(kind)
    bad = table.copy()
    bad[0, 1] = pages.n_pages  # keys 16..31
    cache = pages.to_device(slots)
    out = cache.attend(x, torch.from_numpy(bad).cuda(), lens)
    assert cache.status() == q.ERR_PAGE and "page id" in q.last_error()
    assert cache.status() == q.OK  # read and cleared
    keep = np.r_[0:16, 32:40]
    want, _, size = ref.attention(x[0].double().cpu().numpy(), pages.rows(0, slots)[keep],
                                  pages.rows(1, slots)[keep], 0.125)
    tol, _ = ref.attention_bound(size, 64)
    assert (np.abs(out[0].double().cpu().numpy() - want) <= tol[:, None]).all()
    bad[0, :] = [-1, pages.n_pages, 2 ** 31 - 1, -2 ** 31][:bad.shape[1]]
    out, lse = cache.attend(x, torch.from_numpy(bad).cuda(), lens, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert cache.status() == q.ERR_PAGE


def test_lengths_outside_the_table_are_cut():
    pages, table, slots, x, lens = _small(n=48)
    cache = pages.to_device(slots)
    full = torch.from_numpy(table[:, :3].copy()).cuda()
    want = cache.attend(x, full, lens)
    for n in (49, 2 ** 31 - 1):
        got = cache.attend(x, full, torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert torch.equal(got, want)
        assert cache.status() == q.ERR_PAGE and "length" in q.last_error()
    got = cache.attend(x, full, torch.tensor([-5], dtype=torch.int32, device="cuda"))
    assert (got == 0).all() and cache.status() == q.ERR_PAGE


def test_cache_past_32_bit_offsets():
    """Rows whose byte offsets pass 2^32 in both buffers."""
    page, heads, D = 256, 8, 128
    n_pages = (1 << 33) // (page * heads * D * 2) + 3
    rng = np.random.default_rng(2)
    shape = (n_pages, heads, page, D)
    k = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    lens = [700, 300]
    ids = [n_pages - 1, 0, n_pages - 2, n_pages // 2 + 1, 1]
    vals = []
    for t in (k, v):
        x = torch.from_numpy(rng.standard_normal((5, heads, page, D)).astype(np.float32)).bfloat16()
        t[torch.tensor(ids)] = x.cuda()
        vals.append(x.double().numpy())
    cache = q.KVCache(q.BF16, n_pages, page, heads, D, k=k, v=v)
    table = torch.tensor([ids[:3], ids[3:] + [-1]], dtype=torch.int32, device="cuda")
    x = torch.from_numpy(rng.standard_normal((2, heads, D)).astype(np.float32)).cuda()
    got = cache.attend(x, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    for b, pick in ((0, [0, 1, 2]), (1, [3, 4])):
        kk, vv = (np.concatenate([a[i].transpose(1, 0, 2) for i in pick])[:lens[b]] for a in vals)
        want, _, size = ref.attention(x[b].double().cpu().numpy(), kk, vv,
                                      float(np.float32(1 / math.sqrt(D))))
        tol, _ = ref.attention_bound(size, D)
        assert (np.abs(got[b].double().cpu().numpy() - want) <= tol[:, None]).all()
    # the same rows through append and read
    slots = torch.tensor([(n_pages - 1) * page + 9, (n_pages // 2) * page], device="cuda")
    new = torch.from_numpy(rng.standard_normal((2, heads, D)).astype(np.float32)).bfloat16().cuda()
    cache.append(new, -new, slots)
    rk, rv = cache.read(slots, torch.bfloat16)
    assert torch.equal(rk, new) and torch.equal(rv, -new)
    assert cache.status() == q.OK


def test_bitwise_repeatable():
    rng = np.random.default_rng(4)
    lens = [4001, 17, 0, 950]
    table, n_pages, slots = ref.table_for(lens, 16, rng)
    cache = ref.Pages(q, "bf16", n_pages, 16, 4, 128, rng).to_device(np.concatenate(slots))
    x = torch.from_numpy(rng.standard_normal((4, 16, 128)).astype(np.float32)).cuda()
    t, n = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = cache.attend(x, t, n)
    for _ in range(20):
        assert torch.equal(cache.attend(x, t, n), first)


def test_graph_serves_growing_lengths_and_another_stream():
    rng = np.random.default_rng(6)
    table, n_pages, slots = ref.table_for([600, 600], 16, rng)
    cache = ref.Pages(q, "f16", n_pages, 16, 2, 64, rng).to_device(np.concatenate(slots))
    x = torch.from_numpy(rng.standard_normal((2, 8, 64)).astype(np.float32)).cuda()
    t = torch.from_numpy(table).cuda()
    n = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    cache.attend(x, t, n, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend(x, t, n, out=out)
    side = torch.cuda.Stream()
    for lens in ([1, 0], [17, 400], [600, 3], [0, 0]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        torch.cuda.synchronize()
        direct = cache.attend(x, t, n, stream=side)
        side.synchronize()
        assert torch.equal(direct, replayed), lens


def test_refusals():
    pages, table, slots, x, lens = _small()
    cache = pages.to_device(slots)
    t = torch.from_numpy(table).cuda()
    vp = ctypes.c_void_p
    L = q.lib()
    d = q.AttnDesc(0.1, 0.0, 0, None)

    def call(dtype=q.F32, n=1, heads=4, qp=x.data_ptr(), ldq=256, tp=t.data_ptr(), ldt=t.shape[1],
             lp=lens.data_ptr(), desc=d, op=x.data_ptr(), ldo=256):
        before = q.launch_count()
        rc = L.qmm_attn_decode(cache.h, dtype, n, heads, vp(qp), ldq, vp(tp), ldt, vp(lp),
                               ctypes.byref(desc) if desc else None, vp(op), ldo, None, None)
        assert rc == q.OK or q.launch_count() == before  # a refused call launches nothing
        return rc

    assert call(dtype=8) == q.ERR_FORMAT and "type 8" in q.last_error()
    assert call(heads=3) == q.ERR_SHAPE and "n_q_heads = 3" in q.last_error()
    assert call(heads=0) == q.ERR_SHAPE
    assert call(n=-1) == q.ERR_SHAPE and call(n=0) == q.OK
    assert call(qp=0) == q.ERR_NULL and "q is NULL" in q.last_error()
    assert call(op=0) == q.ERR_NULL and call(tp=0) == q.ERR_NULL and call(lp=0) == q.ERR_NULL
    assert call(desc=None) == q.ERR_NULL
    assert call(qp=x.data_ptr() + 4) == q.ERR_ALIGN and call(ldq=258) == q.ERR_ALIGN
    assert call(ldq=252) == q.ERR_SHAPE and call(ldt=0) == q.ERR_SHAPE
    assert call(desc=q.AttnDesc(math.nan, 0.0, 0, None)) == q.ERR_SHAPE
    assert call(desc=q.AttnDesc(0.1, -1.0, 0, None)) == q.ERR_SHAPE
    assert call(desc=q.AttnDesc(0.1, math.inf, 0, None)) == q.ERR_SHAPE
    assert call(desc=q.AttnDesc(0.1, 0.0, -1, None)) == q.ERR_SHAPE
    for bad in (dict(lens=lens.long()), dict(page_table=t.long()), dict(q=x[0]),
                dict(q=x.double()), dict(q=x[..., :32])):
        a = dict(q=x, page_table=t, lens=lens)
        a.update(bad)
        with pytest.raises((ValueError, q.QmmError)):
            cache.attend(**a)

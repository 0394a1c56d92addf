"""Infinities where the decode attention's formula still has an answer."""
from __future__ import annotations

import math

import numpy as np
import pytest

from tests import _decode_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("before,beside,where", [
    (1e-3, 100.0, 901), (1e-3, 60000.0, 901), (1e-6, 1.0, 901), (2.0, 3.0, 901), (1e-6, 1e-6, 901),
    (1e-6, 1e-6, 3), (1e-3, 2.0, 3), (0.0, 1.0, 3)])
def test_infinite_value_scale_beside_large_ones(D, group, before, beside, where):
    """One block of one key's value has an infinite scale.  The other blocks'
    outputs are what they are without it, also where the keys next to it have
    larger scales than any before."""
    rng = np.random.default_rng(D + group)
    n, B = 1000, 160  # (enough items for a warp to take several tiles of each)
    table, n_pages, slots = ref.table_for([n], 16, rng)
    pages = ref.Pages(q, "q8_0", n_pages, 16, 1, D, rng)
    codes, scales = pages.raw[1]
    at = [(s // 16, 0, s % 16) for s in slots[0]]
    for j, key in enumerate(at):
        scales[key][:D // 32] = np.float16(before if j < 896 else beside)
    scales[at[where]][1] = np.inf
    with np.errstate(invalid="ignore"):
        pages.val[1] = codes.astype(np.float64) * np.repeat(
            scales[..., :D // 32].astype(np.float64), 32, axis=-1)
    cache = pages.to_device(slots[0])
    x = rng.standard_normal((B, group, D)).astype(np.float32)
    scale = float(np.float32(1 / math.sqrt(D)))
    got = cache.attend(torch.from_numpy(x).cuda(), torch.from_numpy(table).cuda().repeat(B, 1),
                       torch.full((B,), n, dtype=torch.int32, device="cuda"), scale=scale)
    got = got.double().cpu().numpy()
    k, v = pages.rows(0, slots[0]), pages.rows(1, slots[0])
    hit = np.zeros(D, bool)
    hit[32:64] = True
    plain = np.where(hit, 0.0, v)
    for b in range(0, B, 40):
        with np.errstate(invalid="ignore"):
            want, _, _ = ref.attention(x[b].astype(np.float64), k, v, scale)
        _, _, size = ref.attention(x[b].astype(np.float64), k, plain, scale)
        tol, _ = ref.attention_bound(size, D)
        assert (np.abs(got[b] - want)[:, ~hit] <= tol[:, None]).all()
        # infinite, or NaN for code 0
        assert np.array_equal(got[b][:, hit], want[:, hit], equal_nan=True)
    cache.close()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("group", [3, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_infinite_query_under_a_cap(kind, group, D):
    """cap * tanh of an infinite score is the cap: an infinite component of q
    gives finite outputs, a NaN stays NaN, and neither touches other heads."""
    rng = np.random.default_rng(group)
    n, cap = 150, 5.0
    table, n_pages, slots = ref.table_for([n], 16, rng)
    pages = ref.Pages(q, kind, n_pages, 16, 1, D, rng)
    if kind == "q8_0":  # (0 times infinity is NaN)
        codes, scales = pages.raw[0]
        codes[codes == 0] = 1
        pages.val[0] = codes.astype(np.float64) * np.repeat(
            scales[..., :D // 32].astype(np.float64), 32, axis=-1)
    cache = pages.to_device(slots[0])
    x = rng.standard_normal((1, group, D)).astype(np.float32)
    x[0, 0, 7], x[0, 1, 33], x[0, 2, 40] = np.inf, -np.inf, np.nan
    scale = float(np.float32(1 / math.sqrt(D)))
    got, lse = cache.attend(torch.from_numpy(x).cuda(), torch.from_numpy(table).cuda(),
                            torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale,
                            softcap=cap, return_lse=True)
    got, lse = got[0].double().cpu().numpy(), lse[0].double().cpu().numpy()
    assert np.isnan(got[2]).all() and np.isnan(lse[2])
    rest = [h for h in range(group) if h != 2]
    k, v = pages.rows(0, slots[0]), pages.rows(1, slots[0])
    with np.errstate(invalid="ignore"):
        want, want_lse, _ = ref.attention(x[0].astype(np.float64), k, v, scale, cap)
    _, _, size = ref.attention(np.where(np.isfinite(x[0]), x[0], 0).astype(np.float64), k, v, scale,
                               cap)
    tol, tol_lse = ref.attention_bound(size, D)
    assert (np.abs(got - want)[rest] <= tol[rest, None]).all()
    assert (np.abs(lse - want_lse)[rest] <= tol_lse[rest]).all()
    # without a cap there is no answer
    got = cache.attend(torch.from_numpy(x).cuda(), torch.from_numpy(table).cuda(),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale)
    assert torch.isnan(got[0, :3]).all() and torch.isfinite(got[0, 3:]).all()
    cache.close()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("group", [1, 4, 8, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,low", [(200, 0), (5000, 2500)])
def test_infinite_value_of_a_key_that_is_never_attended_to(kind, group, D, n, low):
    """A score of -infinity has probability 0, and 0 times infinity is NaN; an
    infinite value elsewhere stays infinite, also of a key (or of `low` keys)
    whose probability is too small for 32 bits."""
    rng = np.random.default_rng(group)
    table, n_pages, slots = ref.table_for([n], 16, rng)
    pages = ref.Pages(q, kind, n_pages, 16, 1, D, rng)
    place = [(s // 16, 0, s % 16) for s in slots[0]]
    dead, far, seen = place[low + 37], place[90], place[low + 151]
    small = place[:low] + [far]
    x = rng.standard_normal((1, group, D)).astype(np.float32)
    x[..., :32] = np.abs(x[..., :32]) + 1
    if kind == "q8_0":
        codes, scales = pages.raw[0]
        codes[dead][:32], scales[dead][0] = -1, np.inf
        for at in small:
            codes[at][:32], scales[at][0] = -127, 60.0
        values, vscales = pages.raw[1]
        for at, block in ((dead, 0), (far, 1)) + ((seen, 1),) * (not low):
            values[at][32 * block:32 * block + 32] = 3
            vscales[at][block] = np.inf
        zero, hit = slice(0, 32), slice(32, 64)
        with np.errstate(invalid="ignore"):
            for w in (0, 1):
                pages.val[w] = pages.raw[w][0].astype(np.float64) * np.repeat(
                    pages.raw[w][1][..., :D // 32].astype(np.float64), 32, axis=-1)
    else:
        k, v = pages.raw[0][0], pages.raw[1][0]
        k[dead] = 0
        k[dead][0] = -math.inf
        for at in small:
            k[at][:32] = -2000.0
        v[dead][5] = v[far][9] = math.inf
        v[seen][9] = 1.0 if low else math.inf  # (with low keys theirs is the only one)
        zero, hit = slice(5, 6), slice(9, 10)
        for w in (0, 1):
            pages.val[w] = pages.raw[w][0].double().numpy()
    cache = pages.to_device(slots[0])
    scale = float(np.float32(1 / math.sqrt(D)))
    got = cache.attend(torch.from_numpy(x).cuda(), torch.from_numpy(table).cuda(),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale)
    got = got[0].double().cpu().numpy()
    assert np.isnan(got[:, zero]).all() and (got[:, hit] == math.inf).all()
    keep = np.ones(D, bool)
    keep[zero] = keep[hit] = False
    sub = np.arange(n) != low + 37
    k, v = pages.rows(0, slots[0])[sub], np.where(keep, pages.rows(1, slots[0])[sub], 0)
    want, _, size = ref.attention(x[0].astype(np.float64), k, v, scale)
    tol, _ = ref.attention_bound(size, D)
    assert (np.abs(got - want)[:, keep] <= tol[:, None]).all()
    cache.close()


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("cap", [1e-30, 1e-39, 1e-45])
def test_caps_of_any_size(kind, cap):
    """A score of 0 stays 0 under a cap whose reciprocal is beyond 32 bits."""
    rng = np.random.default_rng(5)
    n, D = 100, 64
    table, n_pages, slots = ref.table_for([n], 16, rng)
    pages = ref.Pages(q, kind, n_pages, 16, 1, D, rng)
    zero = (slots[0][11] // 16, 0, slots[0][11] % 16)
    pages.raw[0][0][zero] = 0
    pages.val[0][zero] = 0
    cache = pages.to_device(slots[0])
    x = rng.standard_normal((1, 4, D)).astype(np.float32)
    got = cache.attend(torch.from_numpy(x).cuda(), torch.from_numpy(table).cuda(),
                       torch.tensor([n], dtype=torch.int32, device="cuda"), scale=0.125, softcap=cap)
    want, _, size = ref.attention(x[0].astype(np.float64), pages.rows(0, slots[0]),
                                  pages.rows(1, slots[0]), 0.125, float(np.float32(cap)))
    tol, _ = ref.attention_bound(size, D)
    assert (np.abs(got[0].double().cpu().numpy() - want) <= tol[:, None]).all()
    cache.close()

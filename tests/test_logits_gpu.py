"""Penalties, biases and masks on logits (qmm_logits_adjust).  Every step is
one fp32 rounding, so results are compared bit by bit with the same steps
rounded in numpy's float32; odd sizes, misaligned and strided rows, rows
without history, tokens named twice, ids outside the vocabulary."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

from tests import _decode_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")


def bits_of(masks):
    words = (masks.shape[1] + 31) // 32
    padded = np.zeros((masks.shape[0], words * 32), np.uint8)
    padded[:, :masks.shape[1]] = masks
    return np.packbits(padded, axis=1, bitorder="little").view(np.int32)


def same(a, b):
    a, b = np.asarray(a), np.asarray(b)
    return np.array_equal(a, b, equal_nan=True)


def run(B, V, io="f32", history=40, biases=7, masked=True, seed=0, lead=0, gap=0, twice=False,
        in_place=False, shared_mask=False, out_gap=None):
    rng = np.random.default_rng(seed)
    dt = ref.TORCH_IO[io]
    wide = V + lead + gap
    base = torch.from_numpy((3 * rng.standard_normal((B, wide))).astype(np.float32)).to(dt).cuda()
    z = base[:, lead:lead + V]
    host = z.float().cpu().numpy()
    hist = [[int(t) for t in np.where(rng.random(n) < 0.1, -1, (rng.random(n) ** 3 * (V + 2)).astype(int))]
            for n in (rng.integers(0, history + 1, B) if history else [0] * B)]
    bias = [[(int(rng.integers(0, V if not twice else min(V, 5))), float(np.float32(rng.standard_normal())))
             for _ in range(int(rng.integers(0, biases + 1)) if biases else 0)] for _ in range(B)]
    if biases:
        bias[0] += [(-1, 5.0), (V, 5.0), (2 ** 31 - 1, 5.0)]
    masks = rng.random((1 if shared_mask else B, V)) < 0.5
    if not shared_mask and B > 2:
        masks[2] = False
    r, p, f = (rng.uniform(lo, hi, B).astype(np.float32) for lo, hi in ((0.7, 1.4), (-0.5, 1), (-0.2, 0.4)))

    def offs(x):
        return torch.tensor(np.concatenate([[0], np.cumsum([len(i) for i in x])]), device="cuda")

    flat_b = [e for row in bias for e in row]
    out = None
    if in_place:
        out = z
    elif out_gap is not None:
        out = torch.full((B, V + out_gap), 9.0, dtype=dt, device="cuda")[:, :V]
    got = q.logits_adjust(
        z, out, history=torch.tensor([t for row in hist for t in row], dtype=torch.int32, device="cuda"),
        history_offsets=offs(hist), repeat=torch.from_numpy(r).cuda(),
        presence=torch.from_numpy(p).cuda(), frequency=torch.from_numpy(f).cuda(),
        bias_ids=torch.tensor([e[0] for e in flat_b], dtype=torch.int32, device="cuda"),
        bias_values=torch.tensor([e[1] for e in flat_b], dtype=torch.float32, device="cuda"),
        bias_offsets=offs(bias), mask=torch.from_numpy(bits_of(masks)).cuda() if masked else None)
    got = got.cpu()
    for b in range(B):
        want = ref.logits(host[b], hist[b], r[b], p[b], f[b], bias[b],
                          masks[0 if shared_mask else b] if masked else None, dtype=np.float32)
        assert same(got[b].float(), torch.from_numpy(want).to(dt).float()), b


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 32, 33, 1000, 2047, 2048, 2049, 8193, 32003])
@pytest.mark.parametrize("B", [1, 4])
def test_vocabulary_sizes(B, V):
    run(B, V, seed=V)


@pytest.mark.parametrize("io", ["f16", "bf16"])
@pytest.mark.parametrize("V", [7, 4097])
def test_types(io, V):
    run(3, V, io=io, seed=V)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("lead,gap,out_gap", [(1, 0, None), (3, 2, None), (2, 6, 0), (0, 4, 4), (1, 3, 8)])
def test_rows_at_any_place(io, lead, gap, out_gap):
    run(5, 3001, io=io, lead=lead, gap=gap, out_gap=out_gap, seed=lead)


@pytest.mark.parametrize("history,biases,masked", [(0, 0, False), (0, 0, True), (30, 0, False),
                                                   (0, 9, False), (5000, 300, True)])
def test_parts(history, biases, masked):
    run(3, 5003, history=history, biases=biases, masked=masked)


def test_tokens_named_twice_add_in_list_order():
    run(4, 4099, biases=700, twice=True)
    run(3, 5, biases=40, twice=True)


def test_in_place_and_shared_mask():
    run(4, 2050, in_place=True)
    run(4, 2050, shared_mask=True, lead=3)


def test_many_rows_and_long_chunks():
    run(700, 9001, history=20, seed=1)


def test_infinities_nans_and_an_empty_mask():
    V = 70
    z = torch.zeros(3, V, device="cuda")
    z[:, 0], z[:, 1], z[:, 2] = math.nan, math.inf, -math.inf
    masks = np.zeros((3, V), bool)
    masks[1, :] = True
    masks[2, 5:] = True
    ids = torch.tensor([0, 1, 2, 3, 3], dtype=torch.int32, device="cuda")
    out = q.logits_adjust(z, history=ids, history_offsets=torch.tensor([0, 0, 5, 5], device="cuda"),
                          repeat=torch.full((3,), 2.0, device="cuda"),
                          bias_ids=ids[:1], bias_values=torch.tensor([-math.inf], device="cuda"),
                          bias_offsets=torch.tensor([0, 0, 0, 1], device="cuda"),
                          mask=torch.from_numpy(bits_of(masks)).cuda()).cpu()
    assert (out[0] == -math.inf).all()  # what a mask forbids is -inf whatever it was
    assert math.isnan(out[1, 0]) and out[1, 1] == math.inf and out[1, 2] == -math.inf
    assert (out[1, 3:] == 0).all()
    assert (out[2, :5] == -math.inf).all() and (out[2, 5:] == 0).all()


def test_one_row_and_defaults():
    z = torch.randn(501, device="cuda")
    assert torch.equal(q.logits_adjust(z), z)
    h = torch.tensor([4, 4, 500], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 3], device="cuda")
    got = q.logits_adjust(z, history=h, history_offsets=off,
                          frequency=torch.tensor([0.5], device="cuda"))
    want = z.clone()
    want[4] -= 1.0
    want[500] -= 0.5
    assert torch.equal(got, want)
    assert torch.equal(q.logits_adjust(z, history=h, history_offsets=off), z)  # no penalty named


def test_offsets_outside_their_lists_are_clamped():
    z = torch.randn(3, 50, device="cuda")
    h = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    one = torch.ones(3, device="cuda")
    got = q.logits_adjust(z, history=h, presence=one,
                          history_offsets=torch.tensor([-9, 1, 0, 2 ** 40], device="cuda"))
    want = z.clone()
    want[0, 1] -= 1  # [0, 1); then [1, 0) is empty; then [0, 3)
    want[2, 1:4] -= 1
    assert torch.equal(got, want)


def test_refusals():
    z = torch.randn(2, 100, device="cuda")
    L, vp, p = q.lib(), ctypes.c_void_p, z.data_ptr()

    def call(dtype=q.F32, B=2, V=100, src=p, ld=100, dst=p, ldo=100, **rules):
        r = q.LogitRules(**rules)
        before = q.launch_count()
        rc = L.qmm_logits_adjust(dtype, B, V, vp(src), ld, ctypes.byref(r), vp(dst), ldo, None)
        assert rc == q.OK or q.launch_count() == before
        return rc

    assert call(dtype=2) == q.ERR_FORMAT and call(B=-1) == q.ERR_SHAPE and call(B=0) == q.OK
    assert call(V=0) == q.ERR_SHAPE and call(V=2 ** 26 + 1) == q.ERR_SHAPE
    assert call(ld=99) == q.ERR_SHAPE and call(ldo=104) == q.ERR_SHAPE
    assert call(src=0) == q.ERR_NULL and call(dst=0) == q.ERR_NULL
    assert call(src=p + 2) == q.ERR_ALIGN
    assert call(n_history=3) == q.ERR_NULL and "history is NULL" in q.last_error()
    assert call(n_biases=3, bias_ids=p) == q.ERR_NULL and call(n_history=-1) == q.ERR_SHAPE
    assert call(mask=p, ld_mask=3) == q.ERR_SHAPE and "mask" in q.last_error()
    assert call(mask=p + 1, ld_mask=4) == q.ERR_ALIGN
    assert L.qmm_logits_adjust(q.F32, 2, 100, vp(p), 100, None, vp(p), 100, None) == q.ERR_NULL
    for bad in (dict(mask=torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
                dict(repeat=torch.ones(3, device="cuda")), dict(out=z[:1]),
                dict(history=torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            q.logits_adjust(z, **bad)

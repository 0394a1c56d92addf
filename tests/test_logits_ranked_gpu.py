"""qmm_logits_adjust where a block counts the named tokens of its part by their
rank (parts of more than 1024 logits, as large batches get them), also with
more named tokens than are counted at once: every type, in place, a shared
mask, rows at any place, tokens named twice.  Bit by bit against the same steps
in numpy's float32.  That these sizes come to that form is checked in
tests/test_logits_plans.py."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _decode_ref as ref

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")

# rows, vocabulary, type
SIZES = [(700, 9001, "f32"), (760, 12000, "f16"), (380, 20011, "bf16"), (256, 40009, "f32"),
         (8, 400000, "bf16")]
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def packed(masks):
    words = (masks.shape[1] + 31) // 32
    padded = np.zeros((masks.shape[0], words * 32), np.uint8)
    padded[:, :masks.shape[1]] = masks
    return np.packbits(padded, axis=1, bitorder="little").view(np.int32)


def ragged(rng, B, most, draw):
    """Rows of up to `most` entries, row 0 full and row 1 empty, and their offsets."""
    n = rng.integers(0, most + 1, B)
    n[0], n[1] = most, 0
    return draw(int(n.sum())), np.concatenate([[0], np.cumsum(n)])


def check(B, V, io, history=3000, biases=50, twice=False, in_place=False, shared=False, masked=True,
          lead=0, gap=0, seed=0):
    rng = np.random.default_rng(seed + V)
    dt = ref.TORCH_IO[io]
    base = torch.from_numpy((3 * rng.standard_normal((B, V + lead + gap))).astype(np.float32))
    z = base.to(dt).cuda()[:, lead:lead + V]
    host = z.float().cpu().numpy()
    said, h_at = ragged(rng, B, history, lambda n: rng.integers(-1, V + 2, n).astype(np.int32))
    few = min(V, 40)  # tokens that a list with repetitions names
    ids, b_at = ragged(rng, B, biases, lambda n: (
        rng.integers(0, few, n) * (V // few) if twice else rng.integers(-1, V + 1, n)).astype(np.int32))
    values = rng.standard_normal(len(ids)).astype(np.float32)
    masks = rng.random((1 if shared else B, V)) < 0.7
    r, p, f = (rng.uniform(lo, hi, B).astype(np.float32)
               for lo, hi in ((0.7, 1.4), (-0.5, 1), (-0.2, 0.4)))
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    got = q.logits_adjust(z, z if in_place else None, history=dev(said), history_offsets=dev(h_at),
                          repeat=dev(r), presence=dev(p), frequency=dev(f), bias_ids=dev(ids),
                          bias_values=dev(values), bias_offsets=dev(b_at),
                          mask=dev(packed(masks)[0] if shared else packed(masks)) if masked else None)
    got = got.float().cpu().numpy()
    for b in sorted({0, 1, B - 1} | set(range(2, B, max(1, B // 12)))):
        lo, hi = b_at[b], b_at[b + 1]
        want = ref.logits(host[b], said[h_at[b]:h_at[b + 1]], r[b], p[b], f[b],
                          list(zip(ids[lo:hi].tolist(), values[lo:hi])),
                          masks[0 if shared else b] if masked else None, dtype=np.float32)
        want = torch.from_numpy(want).to(dt).float().numpy()
        assert np.array_equal(got[b], want), (b, int((got[b] != want).sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("B,V,io", SIZES)
def test_long_histories(B, V, io):
    check(B, V, io)


@pytest.mark.gpu
@pytest.mark.parametrize("B,V,io", SIZES)
def test_in_place(B, V, io):
    check(B, V, io, in_place=True, seed=1)
    check(B, V, io, in_place=True, masked=False, lead=3, gap=1, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("B,V,io", SIZES)
@pytest.mark.parametrize("lead,gap", [(0, 0), (1, 2), (3, 8)])
def test_shared_mask_and_rows_at_any_place(B, V, io, lead, gap):
    check(B, V, io, shared=True, lead=lead, gap=gap, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("B,V,io", SIZES)
@pytest.mark.parametrize("biases", [3, 300, 3000])
def test_tokens_named_twice(B, V, io, biases):
    check(B, V, io, history=500, biases=biases, twice=True, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("B,V,io", SIZES)
def test_lists_of_one_kind(B, V, io):
    check(B, V, io, history=0, biases=4000, seed=5)
    check(B, V, io, history=2500, biases=0, masked=False, seed=6)

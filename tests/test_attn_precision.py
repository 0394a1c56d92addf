"""How near the decode attention is to 64 bits, by root mean squares over many
scores and outputs (tests/_attn_pieces.py).  On the CPU: the bounds hold for the
arithmetic as the kernels have it and fail once a piece of q or of the
probabilities, the smallest ones of bf16 too, is left out.

A score is a sum of D products.  In fp32 its error is a few roundings of partial
sums, each at most half a unit in the last place of sum |q k|: SCORE such units,
2^-24 of sum |q k|, as a root mean square.  An output adds the errors of its
probabilities (their score's, about two units at these sizes, and the
exponential's two) with random signs, and a few roundings: OUT units of
sum p |v|."""
from __future__ import annotations

import math

import numpy as np
import pytest

from tests import _attn_pieces as ap
from tests import _decode_ref as ref

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")

KINDS = ["f16", "bf16", "q8_0"]
UNIT = 2.0 ** -24
SCORE, OUT = 1.0, 5.0


def one_large(rng, shape):
    """Q8_0 codes as an outlier channel leaves them: it sets each block's scale,
    and the others are small."""
    c = rng.integers(-3, 4, shape)
    c[..., ::32] = 127
    return c.astype(np.int8)


def restated(kind, D, n, q_pieces, p_pieces, offset=0, outlier=False):
    """Errors in units: of the log-sum-exp (the score, for one key), of the outputs."""
    rng = np.random.default_rng(D + n)
    scale = float(np.float32(1 / math.sqrt(D)))
    codes = (lambda r, n, D: one_large(r, (n, D))) if outlier else None
    lse, out, dots, sizes = [], [], [], []
    for _ in range(150):
        keys = ap.Keys(kind, n, D, rng, codes)
        x = rng.standard_normal(D).astype(np.float32)
        if outlier:
            x[::32] *= np.float32(2.0 ** -10)
        got, got_lse = ap.attention(x, keys, scale, q_pieces, p_pieces, offset)
        want, want_lse, dot, size = ap.exact(x, keys, scale)
        lse.append(got_lse - want_lse)
        out.append(got - want)
        dots.append(dot.max())
        sizes.append(size)
    return ap.rms(lse) / ap.rms(dots) / UNIT, ap.rms(out) / ap.rms(sizes) / UNIT


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bounds_tell_a_piece_that_is_missing(kind, D):
    of_q, of_p = ap.PIECES[kind]
    assert restated(kind, D, 1, of_q, of_p)[0] <= SCORE
    assert restated(kind, D, 4, of_q, of_p)[1] <= OUT
    assert restated(kind, D, 1, of_q - 1, of_p)[0] > SCORE
    assert restated(kind, D, 4, of_q, of_p - 1)[1] > OUT


@pytest.mark.parametrize("D", [64, 128, 256])
def test_bounds_tell_codes_that_are_biased_through_the_sums(D):
    assert restated("q8_0", D, 1, 2, 2, outlier=True)[0] <= SCORE
    assert restated("q8_0", D, 1, 2, 2, offset=128, outlier=True)[0] > SCORE


def measured(kind, D, group, n, outlier=False, B=64, H=2):
    rng = np.random.default_rng(1000 * n + D + group)
    table, n_pages, slots = ref.table_for([n] * B, 16, rng)
    pages = ref.Pages(q, kind, n_pages, 16, H, D, rng)
    if outlier:
        codes, scales = pages.raw[0]
        codes[:] = one_large(rng, codes.shape)
        pages.val[0] = codes.astype(np.float64) * np.repeat(
            scales[..., :D // 32].astype(np.float64), 32, axis=-1)
    x = rng.standard_normal((B, H * group, D)).astype(np.float32)
    if outlier:
        x[..., ::32] *= np.float32(2.0 ** -10)
    scale = float(np.float32(1 / math.sqrt(D)))
    cache = pages.to_device(np.concatenate(slots))
    out, lse = cache.attend(torch.from_numpy(x).cuda(), torch.from_numpy(table).cuda(),
                            torch.full((B,), n, dtype=torch.int32, device="cuda"), scale=scale,
                            return_lse=True)
    assert cache.status() == q.OK
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    cache.close()
    errors = [[], [], [], []]
    for b in range(B):
        k, v = pages.rows(0, slots[b]), pages.rows(1, slots[b])
        for h in range(H * group):
            kh, vh = k[:, h // group], v[:, h // group]
            s = kh @ x[b, h].astype(np.float64) * scale
            p = np.exp(s - s.max())
            want = s.max() + math.log(p.sum())
            p /= p.sum()
            errors[0].append(lse[b, h] - want)
            errors[1].append(out[b, h] - p @ vh)
            errors[2].append((np.abs(kh) @ np.abs(x[b, h]).astype(np.float64) * scale).max())
            errors[3].append(p @ np.abs(vh))
    lse, out, dots, sizes = map(ap.rms, errors)
    return lse / dots / UNIT, out / sizes / UNIT


GPU_CASES = [(64, 1), (64, 4), (64, 8), (64, 16), (96, 4), (128, 4), (128, 7), (128, 16), (192, 4),
             (256, 2), (256, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,group", GPU_CASES)
def test_scores(kind, D, group):
    assert measured(kind, D, group, 1)[0] <= SCORE


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,group", GPU_CASES)
def test_outputs(kind, D, group):
    assert measured(kind, D, group, 4)[1] <= OUT


@pytest.mark.gpu
@pytest.mark.parametrize("D,group", GPU_CASES)
def test_scores_of_keys_with_an_outlier_channel(D, group):
    assert measured("q8_0", D, group, 1, outlier=True)[0] <= SCORE

"""Plain 64-bit restatements of the decode-step operators, for the tests: the
paged cache's contents as arrays, rotary positions, attention of one new
token, and logit adjustment.  They share no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

TORCH_IO = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# half a unit in the last place, relative
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


class Pages:
    """A cache's two buffers on the device with known values in the slots that
    are filled and NaN in all others."""

    def __init__(self, q, kind, n_pages, page, heads, D, rng):
        self.kind, self.n_pages, self.page, self.heads, self.D = kind, n_pages, page, heads, D
        shape = (n_pages, heads, page)
        self.val, self.raw = [], []
        for _ in range(2):
            if kind == "q8_0":
                sc = (D // 32 + 1) // 2 * 2
                codes = rng.integers(-127, 128, shape + (D,)).astype(np.int8)
                scales = np.full(shape + (sc,), np.nan, np.float16)
                scales[..., :D // 32] = rng.uniform(0.002, 0.02, shape + (D // 32,))
                self.raw.append([codes, scales])
                self.val.append(codes.astype(np.float64) *
                                np.repeat(scales[..., :D // 32].astype(np.float64), 32, axis=-1))
            else:
                x = torch.from_numpy(rng.standard_normal(shape + (D,)).astype(np.float32))
                x = x.to(TORCH_IO[kind])
                self.raw.append([x])
                self.val.append(x.double().numpy())
        self.q_kind = {"q8_0": q.Q8_0, "f16": q.F16, "bf16": q.BF16}[kind]
        self.q = q

    def rows(self, which, slots):
        """[n, heads, D] values of slot numbers."""
        s = np.asarray(slots)
        return self.val[which][s // self.page, :, s % self.page]

    def to_device(self, used):
        """The handle, with every slot that `used` does not list holding NaN
        (Q8_0: NaN scales)."""
        keep = np.zeros(self.n_pages * self.page, bool)
        keep[np.asarray(used, dtype=np.int64)] = True
        keep = keep.reshape(self.n_pages, 1, self.page, 1)
        bufs = []
        for raw in self.raw:
            if self.kind == "q8_0":
                scales = np.where(keep, raw[1], np.float16(np.nan))
                bufs.append(torch.from_numpy(np.concatenate(
                    [raw[0].reshape(-1).view(np.uint8), scales.reshape(-1).view(np.uint8)])).cuda())
            else:
                bufs.append(torch.where(torch.from_numpy(keep), raw[0],
                                        torch.full_like(raw[0], math.nan)).cuda())
        return self.q.KVCache(self.q_kind, self.n_pages, self.page, self.heads, self.D, k=bufs[0],
                              v=bufs[1])


def table_for(lens, page, rng, spare=2, extra_columns=1):
    """Shuffled pages for sequences of these lengths: (page table with -1 where
    no page is needed, number of pages, slots of each sequence)."""
    need = [-(-max(0, n) // page) for n in lens]
    n_pages = sum(need) + spare
    free = rng.permutation(n_pages)
    table = np.full((len(lens), max(need + [1]) + extra_columns), -1, np.int32)
    slots, at = [], 0
    for b, n in enumerate(need):
        table[b, :n] = free[at:at + n]
        at += n
        j = np.arange(max(0, lens[b]))
        slots.append(table[b, j // page].astype(np.int64) * page + j % page)
    return table, n_pages, slots


def attention(q, k, v, scale, softcap=0.0, window=0, slope=None):
    """One sequence: q [heads, D], k, v [n, kv heads, D] in fp64.  Returns out,
    lse, and what the error bound needs: (largest sum |q k| scale, largest
    |score|, largest |v|) of each head."""
    heads, n = q.shape[0], k.shape[0]
    G = heads // k.shape[1]
    out, lse = np.zeros_like(q), np.full(heads, -np.inf)
    size = np.zeros((heads, 3))
    first = max(0, n - window) if window else 0
    if n == 0:
        return out, lse, size
    k, v, j = k[first:], v[first:], np.arange(first, n)
    for h in range(heads):
        kh, vh = k[:, h // G], v[:, h // G]
        s = kh @ q[h] * scale
        dots = np.abs(kh) @ np.abs(q[h]) * abs(scale)
        if softcap:
            s = softcap * np.tanh(s / softcap)
        bias = slope[h] * (j - (n - 1)) if slope is not None else 0 * s
        s = s + bias
        m = s.max()
        p = np.exp(s - m)
        lse[h] = m + math.log(p.sum())
        out[h] = p @ vh / p.sum()
        size[h] = dots.max(), np.abs(s).max() + np.abs(bias).max() + softcap, np.abs(vh).max()
    return out, lse, size


def attention_bound(size, D):
    """Bounds (out per head, lse per head) of an fp32 computation: scores off by
    the rounding of D products and their sum (2^-24 each, and pieces of q good
    to 2^-22 of its largest component) and a few roundings of the score itself
    in base 2; probabilities off by twice that and their exponential's 2^-21."""
    ds = size[:, 0] * (D + 8) * 2.0 ** -23 + size[:, 1] * 2.0 ** -20
    return size[:, 2] * (2 * ds + 2.0 ** -18), ds + 2.0 ** -19


def rotate(x, pos, inv_freq, sections, pairing):
    """x [T, heads, D] fp64, pos [axes, T] int32; angles are fp32 products."""
    x = np.array(x, dtype=np.float64)
    n = 2 * len(inv_freq)
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = (pos.astype(np.float32)[axis] * np.asarray(inv_freq, np.float32)[:, None]).T
    angle = angle.astype(np.float64)[:, None, :]
    c, s = np.cos(angle), np.sin(angle)
    lo = np.arange(n // 2) if pairing == "halves" else 2 * np.arange(n // 2)
    hi = lo + n // 2 if pairing == "halves" else lo + 1
    a, b = x[..., lo].copy(), x[..., hi].copy()
    x[..., lo], x[..., hi] = a * c - b * s, b * c + a * s
    return x


def rotation_bound(x, n_rot, pairing):
    """Cosine and sine within 2^-22, two products and a sum rounded: of |a| + |b|."""
    x = np.abs(np.array(x, dtype=np.float64))
    half = n_rot // 2
    lo = np.arange(half) if pairing == "halves" else 2 * np.arange(half)
    hi = lo + half if pairing == "halves" else lo + 1
    out = np.zeros_like(x)
    both = (x[..., lo] + x[..., hi]) * 2.0 ** -21
    out[..., lo], out[..., hi] = both, both
    return out


def logits(z, history, repeat, presence, frequency, biases, mask, dtype=np.float64):
    """One row, in the given precision, each step rounded once.  history: ids;
    biases: [(id, value)]; mask: bools or None."""
    z = np.array(z, dtype=dtype)
    V = len(z)
    count = np.zeros(V, np.int64)
    for t in history:
        if 0 <= t < V:
            count[t] += 1
    with np.errstate(all="ignore"):
        for t in np.nonzero(count)[0]:
            x = z[t] / dtype(repeat) if z[t] > 0 else z[t] * dtype(repeat)
            z[t] = x - (dtype(presence) + dtype(frequency) * dtype(count[t]))
        sums = {}
        for t, b in biases:
            if 0 <= t < V:
                sums[t] = dtype(b) if t not in sums else dtype(sums[t] + dtype(b))
        for t, b in sums.items():
            z[t] = z[t] + b
    if mask is not None:
        z[~np.asarray(mask)] = -np.inf
    return z

"""The decode attention's arithmetic restated in numpy, with as many pieces of
q and of the probabilities as asked for, and the measure of its error that
tells them apart: root mean squares over many scores and outputs, against 64
bits.  Single worst cases hide a lost low piece behind their bounds."""
from __future__ import annotations

import math

import numpy as np
import torch

F32 = np.float32
# What a form with 16-bit pieces keeps: of q, of the probabilities.
PIECES = {"f16": (2, 2), "bf16": (3, 3), "q8_0": (2, 2)}


def half(x, kind):
    """x (float32) rounded to the operands' type, as float32."""
    if kind == "bf16":
        return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().float().numpy()
    return x.astype(np.float16).astype(F32)


def pieces(x, n, kind):
    out = []
    for _ in range(n):
        p = half(x, kind)
        out.append(p.astype(np.float64))
        x = (x - p).astype(F32)
    return out


class Keys:
    """n keys and values of one head: values (64 bits) and, for Q8_0, codes and
    scales."""

    def __init__(self, kind, n, D, rng, codes=None):
        self.kind, self.raw, self.val = kind, [], []
        for _ in range(2):
            if kind == "q8_0":
                c = rng.integers(-127, 128, (n, D)) if codes is None else codes(rng, n, D)
                s = rng.uniform(0.005, 0.02, (n, D // 32)).astype(np.float16)
                self.raw.append((c.astype(np.int8), s))
                self.val.append(c * np.repeat(s.astype(np.float64), 32, axis=-1))
            else:
                x = half(rng.standard_normal((n, D)).astype(F32), kind)
                self.raw.append((x, None))
                self.val.append(x.astype(np.float64))


def scores(q, keys, scale, n_pieces, offset=0):
    """One head's scores.  offset: what Q8_0's codes are biased by on their way
    through the sums."""
    kind, D = keys.kind, len(q)
    e = 0
    if kind != "bf16":
        e = 13 - math.frexp(float(np.abs(q).max()))[1] + 1
    parts = pieces((q * F32(2.0 ** e)).astype(F32), n_pieces, kind)
    k, s = keys.raw[0]
    k = k.astype(np.float64) + offset
    step = 32 if kind == "q8_0" else D
    total = np.zeros(len(k), F32)
    for d0 in range(0, D, step):
        sums = []
        for p in parts:
            c = np.full(len(k), -offset * sum(x[d0:d0 + step].sum() for x in parts)
                        if p is parts[0] else 0.0, F32)
            for d in range(d0, d0 + step, 16):  # an instruction's sixteen products
                c = (c + k[:, d:d + 16] @ p[d:d + 16]).astype(F32)
            sums.append(c)
        c = sums[-1]
        for x in sums[-2::-1]:
            c = (c + x).astype(F32)
        if kind == "q8_0":
            total = (total.astype(np.float64) + c.astype(np.float64) * s[:, d0 // 32]).astype(F32)
        else:
            total = c
    return (total * F32(scale * 2.0 ** -e)).astype(F32)


def attention(q, keys, scale, q_pieces, p_pieces, offset=0):
    """(out [D], lse) of one head."""
    kind = keys.kind
    s = (scores(q, keys, scale, q_pieces, offset) * F32(1.4426950408889634)).astype(F32)
    m = s.max()
    p = np.exp2((s - m).astype(np.float64)).astype(F32)
    total = F32(0)
    for x in p:
        total = F32(total + x)
    v, vs = keys.raw[1]
    if kind == "q8_0":
        w = (p[:, None] * F32(2.0 ** 10)).astype(F32)
        w = np.repeat((w * vs.astype(F32)).astype(F32), 32, axis=-1)
    else:
        w = np.repeat((p * F32(2.0 ** 14 if kind == "f16" else 1)).astype(F32)[:, None],
                      v.shape[1], axis=-1)
    out = sum((x * v.astype(np.float64)).sum(0) for x in pieces(w, p_pieces, kind)).astype(F32)
    out = out * F32(2.0 ** {"q8_0": -10, "f16": -14, "bf16": 0}[kind]) / total
    return out, (float(m) + math.log2(total)) * math.log(2.0)


def exact(q, keys, scale):
    """(out, lse) in 64 bits, sum |q k| scale of each key, sum p |v| of each dim."""
    k, v = keys.val
    q = q.astype(np.float64)
    s = k @ q * scale
    p = np.exp(s - s.max())
    lse = s.max() + math.log(p.sum())
    p /= p.sum()
    return p @ v, lse, np.abs(k) @ np.abs(q) * scale, p @ np.abs(v)


def rms(x):
    return float(np.sqrt(np.mean(np.square(np.asarray(x, dtype=np.float64)))))

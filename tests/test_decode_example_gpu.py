"""The example model (examples/decode_step.py) against the same model written
plainly in 64 bits: decoded weights, keys and values kept per sequence, causal
attention.  The cache is bf16 here, rounded on both sides."""
from __future__ import annotations

import importlib.util
import math
import os

import numpy as np
import pytest

from tests import _decode_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("decode_step",
                                                  os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm(x):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)


def bf16(x):
    return torch.from_numpy(x).float().bfloat16().double().numpy()


class Plain:
    """One sequence, token by token, in fp64 (cached rows rounded to bf16)."""

    def __init__(self, ex, model, softcap, window):
        self.ex, self.softcap, self.window = ex, softcap, window
        self.w = [{n: m.dequantize().double().cpu().numpy() for n, m in layer.items()}
                  for layer in model.layers]
        self.head = model.head.dequantize().double().cpu().numpy()
        self.emb = model.embedding.double().cpu().numpy()
        self.inv = model.rope.inv_freq.cpu().numpy()
        self.k = [[] for _ in self.w]
        self.v = [[] for _ in self.w]

    def step(self, token, pos):
        ex = self.ex
        x = self.emb[token]
        turn = lambda t: ref.rotate(t[None], np.array([[pos]], np.int32), self.inv,
                                    [len(self.inv)], "halves")[0]
        for i, w in enumerate(self.w):
            h = norm(x)
            qh = turn((w["q"] @ h).reshape(-1, ex.HEAD_DIM))
            self.k[i].append(bf16(turn((w["k"] @ h).reshape(-1, ex.HEAD_DIM))))
            self.v[i].append(bf16((w["v"] @ h).reshape(-1, ex.HEAD_DIM)))
            out, _, _ = ref.attention(qh, np.array(self.k[i]), np.array(self.v[i]),
                                      1 / math.sqrt(ex.HEAD_DIM), self.softcap, self.window)
            x = x + w["o"] @ norm(out.reshape(-1))
            h = norm(x)
            g, u = w["gate"] @ h, w["up"] @ h
            x = x + w["down"] @ norm(g / (1 + np.exp(-g)) * u)
        return self.head @ norm(x) / ex.D_MODEL


@pytest.mark.parametrize("softcap,window", [(0.0, 0), (30.0, 20)])
def test_generation_matches_the_plain_model(ex, softcap, window):
    prompts = [[11, 7, 900, 45, 3] * 8, [4, 8, 15, 16, 23, 42]]
    model = ex.Model(n_pages=32, kind=q.BF16, softcap=softcap, window=window)
    tokens, logits = ex.generate(model, prompts, 6, banned=(0, 31))
    assert model.status() == [q.OK] * ex.LAYERS
    for b, prompt in enumerate(prompts):
        plain = Plain(ex, model, softcap, window)
        mask = np.ones(ex.VOCAB, bool)
        mask[[0, 31]] = False
        for j, t in enumerate(tokens[b][:-1]):
            z = plain.step(t, j)
            if j < len(prompt) - 1:
                continue
            want = ref.logits(z, tokens[b][:j + 1], np.float32(1.2), np.float32(0.1), 0.0, [], mask)
            got = logits[j + 1 - len(prompt)][b].double().cpu().numpy()
            assert np.array_equal(np.isinf(got), ~mask)
            # A cached value may round to the other bf16 neighbour where fp32 and
            # fp64 differ (a relative 2^-8 of one of thousands of values): logits
            # agree to far better than one part in a hundred of their spread.
            assert np.abs(got - want)[mask].max() <= 0.01 * want[mask].std()


def test_cache_types_agree(ex):
    """The 8-bit cache stays near the 16-bit ones over a whole generation."""
    prompts = [[5, 6, 7, 8, 9, 10, 11, 12] * 3]
    first = {}
    for kind in (q.BF16, q.F16, q.Q8_0):
        model = ex.Model(n_pages=8, kind=kind)
        _, logits = ex.generate(model, prompts, 1)
        first[kind] = logits[0].double().cpu()
    spread = first[q.F16].std()
    assert (first[q.BF16] - first[q.F16]).abs().max() <= 0.05 * spread
    assert (first[q.Q8_0] - first[q.F16]).abs().max() <= 0.05 * spread


def test_example_runs(ex, capsys):
    ex.main()
    assert "prompt tokens" in capsys.readouterr().out

"""A small language model decoded with the library: quantized projections, the
paged key-value cache, attention over it, and adjusted logits.

    python examples/decode_step.py

Two layers with seeded random Q4_K weights; two prompts of different lengths
are read in chunks and continued greedily as one batch, each sequence in pages
of its own.  Every step is what a server's step is:

    q, k, v   = projections (qmm_gemv_batched)
    q         = qmm_kv_append: rotate q and k, store k and v in the cache
    attention = qmm_attn_decode over the pages
    output    = projection, feed-forward (gate, up, SwiGLU, down)
    logits    = projection to the vocabulary
    next      = argmax of qmm_logits_adjust (penalties, biases, a mask)

torch supplies memory, norms, residual sums and the argmax.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import quantized_gguf_dequant_gb300 as q  # noqa: E402
from quantized_gguf_dequant_gb300 import synth  # noqa: E402

D_MODEL, D_FF, VOCAB = 512, 1024, 1000
HEADS, KV_HEADS, HEAD_DIM, LAYERS = 8, 2, 64, 2
PAGE = 16
WIDTHS = {"q": (HEADS * HEAD_DIM, D_MODEL), "k": (KV_HEADS * HEAD_DIM, D_MODEL),
          "v": (KV_HEADS * HEAD_DIM, D_MODEL), "o": (D_MODEL, HEADS * HEAD_DIM),
          "gate": (D_FF, D_MODEL), "up": (D_FF, D_MODEL), "down": (D_MODEL, D_FF)}


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Model:
    """Weights as GGUF bytes on the device, and a cache a layer."""

    def __init__(self, n_pages: int, kind: int = q.Q8_0, softcap: float = 0.0, window: int = 0):
        def weight(N, K, seed):
            return q.Matrix(q.Q4_K, N, K, torch.from_numpy(synth.matrix(q.Q4_K, N, K, seed)).cuda())

        gen = torch.Generator(device="cuda")
        gen.manual_seed(5)
        self.embedding = torch.randn(VOCAB, D_MODEL, device="cuda", generator=gen)
        self.layers = [{n: weight(N, K, 100 * i + j) for j, (n, (N, K)) in enumerate(WIDTHS.items())}
                       for i in range(LAYERS)]
        self.head = weight(VOCAB, D_MODEL, 999)
        self.caches = [q.KVCache(kind, n_pages, PAGE, KV_HEADS, HEAD_DIM) for _ in range(LAYERS)]
        half = HEAD_DIM // 2
        inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float32) / half)
        self.rope = q.Rope(inv)
        self.options = {"softcap": softcap, "window": window}

    def step(self, tokens, pos, slots, page_table, lens):
        """Logits [n, VOCAB] of n <= 16 tokens, each at its own position: token
        i attends to the first lens[i] keys of page_table[i] (its own among
        them).  The tokens of a batch are different sequences'; those of a
        prompt's chunk share their pages and see one key more each."""
        n = tokens.numel()
        x = self.embedding[tokens]
        for w, cache in zip(self.layers, self.caches):
            h = norm(x)
            heads = [w[name].gemv_batched(h).view(n, -1, HEAD_DIM) for name in ("q", "k", "v")]
            rotated = cache.append(heads[1], heads[2], slots, q=heads[0], pos=pos, rope=self.rope)
            seen = cache.attend(rotated, page_table, lens, **self.options)
            x = x + w["o"].gemv_batched(norm(seen.view(n, -1)))
            h = norm(x)
            gate, up = w["gate"].gemv_batched(h), w["up"].gemv_batched(h)
            mid = torch.empty_like(gate)
            q.swiglu(gate, up, mid, mid.numel())
            x = x + w["down"].gemv_batched(norm(mid))
        return self.head.gemv_batched(norm(x)) / D_MODEL

    def status(self):
        return [c.status() for c in self.caches]


class Sequence:
    """One sequence's tokens and pages."""

    def __init__(self, prompt, pages):
        self.tokens, self.pages = list(prompt), list(pages)

    def slot(self, j: int) -> int:
        return self.pages[j // PAGE] * PAGE + j % PAGE


def place(sequences, positions):
    """pos, slots, page table and lengths of one token of each (sequence, position)."""
    width = max(len(s.pages) for s in sequences)
    table = [s.pages + [-1] * (width - len(s.pages)) for s in sequences]
    dev = {"device": "cuda"}
    return (torch.tensor(positions, dtype=torch.int32, **dev),
            torch.tensor([s.slot(j) for s, j in zip(sequences, positions)], **dev),
            torch.tensor(table, dtype=torch.int32, **dev),
            torch.tensor([j + 1 for j in positions], dtype=torch.int32, **dev))


def generate(model, prompts, new_tokens: int, chunk: int = 16, banned=()):
    """The prompts' greedy continuations, penalised for repetition and never a
    banned token; also the logits of every generated token."""
    need = [-(-(len(p) + new_tokens) // PAGE) for p in prompts]
    order = iter(reversed(range(sum(need))))  # any pages will do
    sequences = [Sequence(p, [next(order) for _ in range(n)]) for p, n in zip(prompts, need)]
    for s in sequences:  # all but a prompt's last token: only the cache matters
        for a in range(0, len(s.tokens) - 1, chunk):
            at = list(range(a, min(a + chunk, len(s.tokens) - 1)))
            model.step(torch.tensor([s.tokens[j] for j in at], device="cuda"),
                       *place([s] * len(at), at))
    words = [0xffffffff] * ((VOCAB + 31) // 32)
    for t in banned:
        words[t // 32] &= ~(1 << (t % 32))
    allowed = torch.tensor(words, dtype=torch.int64).to(torch.int32).cuda()
    n = len(sequences)
    repeat = torch.full((n,), 1.2, device="cuda")
    presence = torch.full((n,), 0.1, device="cuda")
    every = []
    for _ in range(new_tokens):
        last = [len(s.tokens) - 1 for s in sequences]
        z = model.step(torch.tensor([s.tokens[-1] for s in sequences], device="cuda"),
                       *place(sequences, last))
        said = [t for s in sequences for t in s.tokens]
        ends = torch.tensor([0] + [len(s.tokens) for s in sequences], device="cuda").cumsum(0)
        z = q.logits_adjust(z, history=torch.tensor(said, dtype=torch.int32, device="cuda"),
                            history_offsets=ends, repeat=repeat, presence=presence, mask=allowed)
        every.append(z)
        for s, t in zip(sequences, z.argmax(-1).tolist()):
            s.tokens.append(t)
    return [s.tokens for s in sequences], every


def main():
    prompts = [[11, 7, 900, 45, 3] * 9, [4, 8, 15, 16, 23, 42]]
    model = Model(n_pages=32)
    tokens, _ = generate(model, prompts, 12, banned=(0, 31))
    assert model.status() == [q.OK] * LAYERS
    for p, t in zip(prompts, tokens):
        print(len(p), "prompt tokens, then", t[len(p):])


if __name__ == "__main__":
    main()

"""How qmm_logits_adjust cuts rows into parts (no GPU): every logit in one part,
parts that a block's bitmap holds, and which form the GPU tests' sizes take."""
from __future__ import annotations

import os
import subprocess

import pytest

from quantized_gguf_dequant_gb300 import build as qbuild
from tests import test_logits_ranked_gpu as ranked

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 152


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    qbuild.build()
    objects = [os.path.join(qbuild.BUILD, os.path.splitext(s)[0] + ".o") for s in qbuild.SOURCES]
    if not all(os.path.exists(o) for o in objects):
        qbuild.build(force=True)
    exe = str(tmp_path_factory.mktemp("logits") / "host_logits")
    subprocess.run([qbuild.nvcc(), "-std=c++17", "-O1", "-I" + os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "host_logits.cu"), *objects, "-o", exe,
                    *qbuild.ARCH], check=True, capture_output=True)

    def of(cases):
        args = [str(x) for c in cases for x in c]
        out = subprocess.run([exe, str(SMS), *args], check=True, capture_output=True, text=True)
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]

    return of


def test_the_ranked_tests_sizes_are_ranked(plan):
    plans = plan([(B, V, ranked.BYTES[io]) for B, V, io in ranked.SIZES])
    for (B, V, io), (parts, part, at_once) in zip(ranked.SIZES, plans):
        assert part > at_once, (B, V, io)
        # 3000 tokens drawn from the vocabulary are more than are counted at once
        # in a part of at least half of it
        if parts <= 2:
            assert 3000 / parts * 0.8 > at_once
    assert sum(p[0] <= 2 for p in plans) >= 3


def test_parts_cover_their_rows(plan):
    cases = [(B, V, b) for B in (1, 2, 7, 30, 152, 700, 5000) for b in (2, 4)
             for V in (1, 5, 1000, 1024, 1025, 16384, 16385, 32001, 128256, 262144, 1 << 26)]
    for (B, V, b), (parts, part, _) in zip(cases, plan(cases)):
        n = 16 // b
        assert parts >= 1 and part % n == 0
        assert parts * part >= V + n - 1  # whatever the row's misalignment
        assert part <= 16384 + 2 * n

"""Every kernel of the decode-step operators that is compiled is one that a call
can reach (no GPU: the names of the objects' launch stubs)."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from quantized_gguf_dequant_gb300 import build as qbuild

pytestmark = pytest.mark.skipif(shutil.which("nm") is None, reason="nm lists the kernels")


def stubs(source, pattern):
    qbuild.build()
    path = os.path.join(qbuild.BUILD, source + ".o")
    if not os.path.exists(path):
        qbuild.build(force=True)
    names = subprocess.run(["nm", path], check=True, capture_output=True, text=True).stdout
    return {tuple(map(int, m)) for m in re.findall(pattern, names)}


@pytest.mark.parametrize("source,kind", [("attn_f16", 0), ("attn_bf16", 1), ("attn_q8", 2)])
def test_attention_kernels(source, kind):
    """(kind, head_dim, heads, warps)"""
    want = set()
    for D in (64, 96, 128, 192, 256):
        q8 = kind == 2
        warps = {64: 4 if q8 else 8, 96: 6, 256: 4 if q8 else 6}.get(D, 4)
        heads = [4, 8]
        if (D == 64 and not q8) or (D == 128 and kind == 0):
            heads.append(16)
        for h in heads:
            want.add((kind, D, h, warps))
            if D == 128 and h <= 8:
                want.add((kind, D, h, 12))
    assert stubs(source, r"attn_kernelILN[^E]*KindE(\d)ELi(\d+)ELi(\d+)ELi(\d+)E") == want


def test_append_kernels():
    """(kind, head_dim): head_dim 96 in Q8_0 has no whole blocks on neighbouring
    lanes and takes the general kernel."""
    got = stubs("kv_append", r"append_kernelILN[^E]*KindE(\d)E[^L]*Li(\d+)E")
    assert got == {(k, D) for k in (0, 1, 2) for D in (64, 96, 128, 192, 256)} - {(2, 96)}

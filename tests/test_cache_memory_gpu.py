"""What a cache's handle takes on the device beside its two buffers."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")

MB = 1 << 20


@pytest.mark.parametrize("kind,head_dim,most", [
    ("F16", 64, 2.6), ("BF16", 64, 2.6), ("Q8_0", 64, 2.6), ("F16", 128, 7.6), ("BF16", 128, 3.8),
    ("Q8_0", 128, 3.8), ("F16", 256, 2.6), ("Q8_0", 192, 5.7), ("Q8_0", 256, 5.1)])
def test_workspace(kind, head_dim, most):
    """include/qmm.h names the sizes on 152 SMs; the device gives memory out in
    pieces of 2 MB."""
    n = 32
    q.KVCache(getattr(q, kind), 1, 16, 1, head_dim).close()
    buffers = [torch.zeros(q.kv_bytes(getattr(q, kind), 1, 16, 1, head_dim), dtype=torch.uint8,
                           device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    caches = [q.KVCache(getattr(q, kind), 1, 16, 1, head_dim, *buffers) for _ in range(n)]
    took = (before - torch.cuda.mem_get_info()[0]) / n
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert took <= most * 1e6 * sms / 152 + 2 * MB
    for c in caches:
        c.close()

"""Which type qmm_kv_read's Python call takes where none is named."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")


@pytest.mark.parametrize("given", ["k_out", "v_out"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_the_type_of_the_output_that_is_given(given, dtype):
    cache = q.KVCache(q.F16, 2, 16, 2, 64)
    x = torch.randn(20, 2, 64, device="cuda").half()
    slots = torch.arange(20, device="cuda")
    cache.append(x, -x, slots)
    out = torch.empty(20, 2, 64, dtype=dtype, device="cuda")
    k, v = cache.read(slots, **{given: out})
    assert (k if given == "k_out" else v) is out and k.dtype == v.dtype == dtype
    assert torch.equal(k, x.to(dtype)) and torch.equal(v, (-x).to(dtype))
    cache.close()

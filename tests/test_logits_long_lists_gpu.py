"""qmm_logits_adjust with long bias lists that name tokens again and again: the
sums in list order, in a time that follows the list's length."""
from __future__ import annotations

import numpy as np
import pytest

from tests import _decode_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")


def lists(rng, B, n, tokens):
    ids = rng.integers(0, tokens, (B, n)).astype(np.int32)
    return ids, rng.standard_normal((B, n)).astype(np.float32)


def call(z, ids, values):
    B, n = ids.shape
    return q.logits_adjust(z, bias_ids=ids.view(-1), bias_values=values.view(-1),
                           bias_offsets=torch.arange(0, (B + 1) * n, n, device="cuda"))


@pytest.mark.parametrize("B,V", [(2, 5000), (700, 9001)])
@pytest.mark.parametrize("n,tokens", [(5000, 3), (5000, 4000), (3001, 1)])
def test_sums_in_list_order(B, V, n, tokens):
    rng = np.random.default_rng(n + tokens)
    ids, values = lists(rng, B, n, tokens)
    ids[:, -40:] = rng.integers(-1, V + 1, (B, 40))
    if B > 4:  # one row names nothing twice
        ids[3] = rng.permutation(V)[:n]
    z = rng.standard_normal((B, V)).astype(np.float32)
    got = call(*(torch.from_numpy(x).cuda() for x in (z, ids, values))).cpu().numpy()
    for b in {0, 1, 3 % B, B - 1}:
        want = ref.logits(z[b], [], 1, 0, 0, list(zip(ids[b].tolist(), values[b])), None,
                          dtype=np.float32)
        assert np.array_equal(got[b], want), b


@pytest.mark.parametrize("B,V", [(4, 128256), (256, 40009)])
@pytest.mark.parametrize("repeated", [1, 15000])
def test_time_of_lists_that_name_tokens_twice(B, V, repeated):
    """Adding in list order takes one more pass over the list, by one warp instead
    of the block's eight: ten times as long as the same list without repetitions
    is more than that.  A search from each entry on would take hundreds of times
    as long."""
    rng = np.random.default_rng(1)
    n = 30000
    z = torch.from_numpy(rng.standard_normal((B, V)).astype(np.float32)).cuda()
    took = []
    for names in (n, n - repeated):
        ids = np.stack([np.resize(rng.permutation(V)[:names], n) for _ in range(B)]).astype(np.int32)
        given = torch.from_numpy(ids).cuda(), torch.randn(B, n, device="cuda")
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call(z, *given)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        took.append(sorted(times)[2])
    print("ms:", took)
    assert took[1] <= 10 * took[0]

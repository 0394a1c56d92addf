"""Calls on a stream that is not the current one: what they read may be
dropped by the caller at once."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
q = pytest.importorskip("quantized_gguf_dequant_gb300")

T, HEADS, D, PAGE = 300, 2, 64, 16


def f16(*shape):
    return torch.randn(*shape, device="cuda").half()


def append(cache, stream):
    rope = q.Rope(torch.ones(D // 2, device="cuda"))
    given = [f16(T, HEADS, D), f16(T, HEADS, D), torch.arange(T, device="cuda"), f16(T, 4, D),
             torch.zeros(T, dtype=torch.int32, device="cuda"), f16(T, 4, D)]
    k, v, slots, x, pos, out = given
    stream.wait_stream(torch.cuda.current_stream())
    return given + [rope.inv_freq], lambda on: cache.append(k, v, slots, q=x, pos=pos, rope=rope,
                                                            q_out=out, stream=on)


def attend(cache, stream):
    lens = torch.full((T,), 40, dtype=torch.int32, device="cuda")
    table = torch.arange(3, dtype=torch.int32, device="cuda").repeat(T, 1)
    given = [f16(T, 4, D), table, lens, torch.ones(4, device="cuda"), f16(T, 4, D),
             torch.empty(T * 4, device="cuda")]
    x, _, _, alibi, out, lse = given
    stream.wait_stream(torch.cuda.current_stream())
    return given, lambda on: cache.attend(x, table, lens, alibi=alibi, out=out, lse=lse, stream=on)


def read(cache, stream):
    given = [torch.arange(T, device="cuda"), f16(T, HEADS, D), f16(T, HEADS, D)]
    slots, k, v = given
    stream.wait_stream(torch.cuda.current_stream())
    return given, lambda on: cache.read(slots, torch.float16, k_out=k, v_out=v, stream=on)


def logits(cache, stream):
    B, V = 30, 1000
    said = torch.arange(B, dtype=torch.int32, device="cuda")
    offsets = torch.arange(B + 1, device="cuda")
    given = [f16(B, V), f16(B, V), said, offsets, torch.ones(B, device="cuda"),
             torch.ones(B, device="cuda"), torch.ones(B, device="cuda"), said.clone(),
             torch.ones(B, device="cuda"), offsets.clone(),
             torch.zeros(B, 32, dtype=torch.int32, device="cuda")]
    z, out, h, ho, r, p, f, bi, bv, bo, m = given
    stream.wait_stream(torch.cuda.current_stream())
    return given, lambda on: q.logits_adjust(
        z, out, history=h, history_offsets=ho, repeat=r, presence=p, frequency=f, bias_ids=bi,
        bias_values=bv, bias_offsets=bo, mask=m, stream=on)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("make", [append, attend, read, logits])
def test_inputs_dropped_after_a_call_on_another_stream(make, raw):
    cache = q.KVCache(q.F16, 20, PAGE, HEADS, D)
    side = torch.cuda.Stream()
    given, call = make(cache, side)
    with torch.cuda.stream(side):
        a = torch.zeros(4096, 4096, device="cuda")
        a = a @ a  # (the first product sets its library up)
    on = side.cuda_stream if raw else side
    call(on)  # (a kernel's first launch may wait for the device)
    torch.cuda.synchronize()
    # the stream has much to do before it comes to the call
    with torch.cuda.stream(side):
        for _ in range(60):
            a = a @ a
    call(on)
    busy = not side.query()
    held = [(t.data_ptr(), t.numel() * t.element_size()) for t in given]
    sizes = [n for _, n in held]
    del given, call
    new = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes * 4]
    taken = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in new]
    assert busy  # else the memory was free to be given out
    for at, n in held:
        assert not any(lo < at + n and at < hi for lo, hi in taken)
    torch.cuda.synchronize()
    cache.close()

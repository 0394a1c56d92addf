"""What the Python calls of the decode-step operators refuse before they reach
the C entries, without a GPU (tests/_binding_host.py)."""
from __future__ import annotations

import pytest

import quantized_gguf_dequant_gb300 as q
from quantized_gguf_dequant_gb300 import build as qbuild
from tests import _binding_host as host

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def outcome(tmp_path_factory):
    qbuild.build()
    directory = str(tmp_path_factory.mktemp("binding"))
    host.build(directory)

    def of(name, **args):
        return host.outcomes(directory, [{"name": name, "args": args}])[0]

    return of


def logits(device, **more):
    t = [[2, 100], "f32", device]
    return dict(logits=t, out=t, **more)


def test_logits_of_another_device_than_the_current_one_refuse(outcome):
    assert outcome("logits_adjust", **logits(0)) == "called"
    got = outcome("logits_adjust", **logits(1))
    assert got.startswith("ValueError") and "device 1" in got and "device 0" in got


class Buffer:
    """What KVCache asks of a buffer before it makes a handle."""

    def __init__(self, device):
        self.device = torch.device("cuda", device)
        self.is_cuda = True

    def numel(self):
        return 1 << 20

    def element_size(self):
        return 1


@pytest.mark.parametrize("k,v", [(1, 1), (0, 1), (1, 0)])
def test_cache_buffers_of_another_device_than_the_current_one_refuse(monkeypatch, k, v):
    qbuild.build()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    made = []
    monkeypatch.setattr(q, "_ptr", lambda t: made.append(t))
    with pytest.raises(ValueError, match="device"):
        q.KVCache(q.F16, 2, 16, 2, 64, k=Buffer(k), v=Buffer(v))
    assert not made  # nothing was handed to the library


def rope(device):
    return {"pairs": [32], "device": device}


def new_tokens(device, rope_device):
    t, slots = [[3, 2, 64], "f32", device], [[3], "i64", device]
    return dict(k=t, v=t, slots=slots, q=t, q_out=t, pos=[[3], "i32", device],
                rope=rope(rope_device))


def test_frequencies_of_another_device_refuse(outcome):
    assert outcome("append", **new_tokens(0, 0)) == "called"
    got = outcome("append", **new_tokens(0, 1))
    assert got.startswith("ValueError") and "inv_freq" in got


@pytest.mark.parametrize("pairs,shape,taken", [
    ([16, 16], [2, 3], True), ([16, 16], [3, 2], False), ([16, 16], [6], False),
    ([10, 11, 11], [3, 3], True), ([32], [3], True), ([32], [1, 3], True), ([32], [4], False),
    ([32], [2, 3], False)])
def test_positions_are_taken_by_axis_then_token(outcome, pairs, shape, taken):
    args = new_tokens(0, 0)
    args["rope"]["pairs"], args["pos"] = pairs, [shape, "i32", 0]
    got = outcome("append", **args)
    if taken:
        assert got == "called"
    else:
        assert got.startswith("ValueError") and "pos" in got

"""clip_grads() of a layer whose gradient buffers were replaced or moved, on another stream, and with norms
that are kept. A norm is within 2^-23 of the exact one, a clipped gradient within the roundings of
test_gpu_layer_grouped.py."""
import math

import pytest
import torch

from gpu_util import say
from test_gpu_layer_grouped import _clipped, _mel, _rand

pytestmark = pytest.mark.gpu


def _layer(mel, dtype="bf16"):
    layer = mel.MoELoRALayer(mel.Shape(16, 64, 32, 8, 2, 4, dtype), "softmax_topk")
    for i, g in enumerate(layer.grads.values()):
        g.copy_(_rand(*g.shape, dtype=dtype, seed=i))
    return layer


def _exact(bufs):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in bufs))


@pytest.mark.parametrize("how", ["replaced", "moved"])
def test_other_buffers_than_at_the_first_call(how):
    mel = _mel()
    say(f"[clip_grads] {how}")
    layer = _layer(mel)
    layer.clip_grads(1e9)
    old = layer.grads["db_gu"]
    fresh = _rand(*old.shape, seed=9) * 3
    kept = old.clone()
    if how == "replaced":
        layer.grads["db_gu"] = fresh
    else:
        old_data = old.data
        old.data = fresh
    bufs = layer._grad_buffers()
    before = [g.clone() for g in bufs]
    norm = layer.clip_grads(0.5)
    torch.cuda.synchronize()
    assert layer.grads["db_gu"].data_ptr() == fresh.data_ptr()
    _clipped(bufs, before, norm, 0.5)
    assert torch.equal(old if how == "replaced" else old_data, kept)


def test_norms_that_are_kept():
    mel = _mel()
    say("[clip_grads norms]")
    layer = _layer(mel, "f32")
    norms, exact = [torch.empty(1, device="cuda") for _ in range(3)], []
    for n in norms:
        exact.append(_exact(layer.grads.values()))
        assert layer.clip_grads(exact[-1] / 2, norm=n) is n
        torch.cuda.synchronize()
    for n, e in zip(norms, exact):
        assert abs(float(n) - e) <= 2.0 ** -23 * e
    assert exact[2] < 0.3 * exact[0]
    assert layer.clip_grads(1e9).data_ptr() == layer.clip_grads(1e9).data_ptr()
    with pytest.raises(ValueError):
        layer.clip_grads(1.0, norm=torch.empty(2, device="cuda"))


def stream_of(t):
    """The stream for which torch allocated a tensor's memory."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]


def test_memory_for_the_default_stream_by_its_number():
    mel = _mel()
    say("[clip_grads stream 0]")
    layer = _layer(mel)
    bufs = layer._grad_buffers()
    before = [g.clone() for g in bufs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        norm = layer.clip_grads(0.5, stream=0)
    assert stream_of(norm) == torch.cuda.default_stream().cuda_stream == 0
    torch.cuda.synchronize()
    _clipped(bufs, before, norm, 0.5)


@pytest.mark.parametrize("raw", [False, True])
def test_memory_belongs_to_the_stream_of_the_call(raw):
    mel = _mel()
    say(f"[clip_grads stream] raw={raw}")
    layer = _layer(mel)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    bufs = layer._grad_buffers()
    before = [g.clone() for g in bufs]
    torch.cuda.synchronize()
    norm = layer.clip_grads(0.5, stream=side.cuda_stream if raw else side)
    assert stream_of(norm) == side.cuda_stream
    side.synchronize()
    _clipped(bufs, before, norm, 0.5)

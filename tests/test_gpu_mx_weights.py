"""mx_weights on a stream of the caller's: its results' memory belongs to that stream, and they are the
ones of the current stream."""
import pytest
import torch

from gpu_util import say
from test_gpu_clip_grads import stream_of
from test_gpu_layer_grouped import _mel, _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_on_another_stream(raw):
    mel = _mel()
    say(f"[mx_weights stream] raw={raw}")
    w_gu, w_d = _rand(4, 1024, 512), _rand(4, 512, 512)
    want = mel.mx_weights(w_gu, w_d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    # blocks of the sizes that are needed, free for the current stream
    del_me = [torch.empty_like(v) for v in want.values()]
    del del_me
    got = mel.mx_weights(w_gu, w_d, side.cuda_stream if raw else side)
    assert all(stream_of(v) == side.cuda_stream for v in got.values())
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)

"""Which gradients a layer clips together: those of its weights and vectors, not those that go on to what
computed its inputs. On the CPU: no kernel is launched."""
import pytest

from test_abi_residual import lib  # noqa: F401  (fixture)


@pytest.mark.parametrize("gate,clipped", [("none", False), ("channel", True), ("token", False), ("full", False)])
@pytest.mark.parametrize("shared_I,full_ft", [(None, False), (32, True)])
def test_sublayer(lib, gate, clipped, shared_I, full_ft):  # noqa: F811
    import mixture_experts_lora_amd as mel
    sub = mel.MoELoRASublayer(mel.Shape(16, 64, 32, 8, 2, 4, "bf16"), "softmax_topk", shared_I, attn_width=48,
                              attn_bias=True, post="layer", gate=gate, device="cpu", full_ft=full_ft)
    bufs = {b.data_ptr() for b in sub._grad_buffers()}
    assert ("dgate" in sub.grads) == (gate != "none")
    for n, g in sub.grads.items():
        assert (g.data_ptr() in bufs) == (n != "dgate" or clipped), n
    assert len(sub._grad_buffers()) == len(sub.grads) - (gate in ("token", "full")) + \
        (4 + 2 * full_ft) * (2 if shared_I else 1)
    for act in (sub.dh, sub.dattn, sub.block.routed.dx, sub.block.routed.d_logits):
        assert act.data_ptr() not in bufs

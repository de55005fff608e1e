"""The forward of an exported layer, weights in 4 bits and activations in 8, on the residual stream:
every stage against float64 on what the stage before it left.

The norm's 8-bit rows are the quantised x, code for code. Routing: the oracle's choice, weights to 1e-5.
The products' tolerances are those of the microscaled products. The combine is a float32 sum of k + 1
terms (with a shared expert one more rounding of y) and one rounding, u = eps / 2 of the dtype; the
stream adds h with one more."""
import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import grouped as G
from oracle import microscale as X
from test_gpu_layer_grouped import DT, _rand
from test_gpu_mx_linear import compare, reference

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _merged(E, H, I, dtype, seed=0):
    lead = (E,) if E else ()
    return (_rand(*lead, 2 * I, H, dtype=dtype, std=H ** -0.5, seed=seed),
            _rand(*lead, H, I, dtype=dtype, std=I ** -0.5, seed=seed + 1))


def _values(codes, scales, fmt):
    c, s = codes.cpu().numpy(), scales.cpu().numpy()
    flat = X.unpack(c.reshape(-1, c.shape[-1]), fmt)
    return X.dequantize(flat, s.reshape(-1, s.shape[-1]), fmt).reshape(*c.shape[:-1], -1)


def _sublayer(mel, T, dtype, shared_I=None, E=16, k=4, H=160, I=96, **kw):
    router = mel.GroupedRouter(E, k, groups=4, topk_groups=2, scale=2.5)
    sub = mel.MoEMXSublayer(mel.Shape(T, H, I, E, k, 4, dtype), router, shared_I, **kw)
    w = mel.mx_weights(*_merged(E, H, I, dtype))
    sw = mel.mx_weights(*_merged(0, H, shared_I, dtype, seed=5)) if shared_I else None
    prm = {n: 1 + _rand(*s, dtype=dtype, std=0.1) for n, s in sub.param_shapes().items()}
    x = dict(h=_rand(T, H, dtype=dtype), w_r=_rand(E, H, dtype=dtype, std=H ** -0.5),
             bias=_rand(E, dtype="f32", std=0.1))

    def run(stream=None):
        return sub.forward(x["h"], prm, x["w_r"], w, sw, stream, x["bias"])

    return sub, run, x, w, sw


@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shared_I", [None, 64])
def test_stages(T, dtype, shared_I):
    mel = _mel()
    say(f"[exported layer] T={T} {dtype} shared={shared_I}")
    sub, run, x, w, sw = _sublayer(mel, T, dtype, shared_I)
    run()
    torch.cuda.synchronize()
    L, s = sub.layer, sub.shape
    u = torch.finfo(DT[dtype]).eps / 2
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    codes, scales = X.quantize(f64(sub.x), "fp8")
    assert (X.pack(codes, "fp8") == L.x_codes.cpu().numpy()).all()
    assert (scales == L.x_scales.cpu().numpy()).all()
    logits = f64(sub.logits)
    ids = G.choose(logits, s.k, "sigmoid", 4, 2, 2, f64(x["bias"]))
    assert (ids == L.topk_ids.cpu().numpy()).all()
    rw = G.weights(logits, ids, "sigmoid", True, 2.5)
    assert np.abs(f64(L.topk_w) - rw).max() <= 1e-5 * rw.max()
    # the experts
    rows, offsets = L.sorted_pair.cpu().numpy(), L.offsets.cpu().numpy()
    a = _values(L.x_codes, L.x_scales, "fp8")
    up, down = _values(w["w_gu"], w["s_gu"], "fp4"), _values(w["w_d"], w["s_d"], "fp4")
    compare("mx8", L.experts.act, L.experts.act_scales, *reference(a[rows // s.k], up, offsets, s.N, True))
    act = _values(L.experts.act, L.experts.act_scales, "fp8")
    compare(dtype, L.y_exp, None, *reference(act, down, offsets, s.N, False))
    # combine, shared expert, stream
    terms = f64(L.y_exp)[L.inv_pos.cpu().numpy()].reshape(T, s.k, s.H) * f64(L.topk_w)[..., None]
    y, size = terms.sum(1), np.abs(terms).sum(1)
    err = u * np.abs(y) + (s.k + 1) * E24 * size
    if shared_I:
        compare("mx8", L.shared.act, L.shared.act_scales,
                *reference(a, _values(sw["w_gu"], sw["s_gu"], "fp4"), None, T, True))
        act = _values(L.shared.act, L.shared.act_scales, "fp8")
        compare(dtype, L.shared_y, None,
                *reference(act, _values(sw["w_d"], sw["s_d"], "fp4"), None, T, False))
        y = y + f64(L.shared_y)
        err = err * (1 + u) + (u + E24) * np.abs(y)
    assert (np.abs(f64(L.y) - y) <= err + 1e-7).all()
    got, ref = f64(sub.h2), f64(x["h"]) + f64(L.y)
    assert (np.abs(got - ref) <= (u + 4 * E24) * np.abs(ref) + 4 * E24 * np.abs(f64(x["h"])) + 1e-7).all()


@pytest.mark.parametrize("T", [1, 130])
def test_captured_and_on_a_stream(T):
    mel = _mel()
    say(f"[exported layer captured] T={T}")
    sub, run, x, _, _ = _sublayer(mel, T, "bf16", 64, post="rms", gate="token", gate_sigmoid=True)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    side = torch.cuda.Stream()
    for i in range(4):
        x["h"].copy_(_rand(*x["h"].shape, seed=30 + i))
        sub.h2.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = sub.h2.clone()
        sub.h2.zero_()
        torch.cuda.synchronize()
        run(stream=side)
        side.synchronize()
        assert torch.equal(got, sub.h2), i


def test_layers_of_other_lengths_share_weights():
    """A prefill's rows and each of them alone: the same results where the same kernel takes them, and
    always the same routing and codes."""
    mel = _mel()
    E, k, H, I = 8, 2, 128, 64
    router = mel.GroupedRouter(E, k, score="softmax")
    w = mel.mx_weights(*_merged(E, H, I, "bf16"))
    x, logits = _rand(6, H), _rand(6, E, dtype="f32")
    whole = mel.MoEMXLayer(mel.Shape(6, H, I, E, k, 4), router)
    y = whole.forward(x, logits, w)
    one = mel.MoEMXLayer(mel.Shape(1, H, I, E, k, 4), router)
    for t in range(6):
        got = one.forward(x[t:t + 1].clone(), logits[t:t + 1].clone(), w)
        torch.cuda.synchronize()
        assert torch.equal(one.topk_ids[0], whole.topk_ids[t])
        assert torch.equal(one.x_codes[0], whole.x_codes[t])
        assert torch.equal(got[0], y[t])


def test_refusals():
    mel = _mel()
    with pytest.raises(ValueError, match="bf16 or f16"):
        mel.MoEMXLayer(mel.Shape(4, 64, 32, 8, 2, 4, "f32"), mel.GroupedRouter(8, 2))
    with pytest.raises(RuntimeError, match="multiple of 32"):
        mel.MoEMXLayer(mel.Shape(4, 48, 32, 8, 2, 4), mel.GroupedRouter(8, 2))
    with pytest.raises(ValueError, match="norm"):
        mel.MoEMXSublayer(mel.Shape(4, 64, 32, 8, 2, 4), mel.GroupedRouter(8, 2), norm="none")

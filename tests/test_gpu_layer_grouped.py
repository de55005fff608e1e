"""Layers that route by groups with a balance bias, and the clipping of their gradients.

The layer's routing is compared to the float64 oracle (weights to 1e-5, as for the other modes). With
the choice held fixed, dL = sum <dy, y> depends on the logits through the weights alone, so d logits is
compared to central differences of sum w_tj <dy_t, y_exp_tj> with float64 weights (step 1e-4: truncation
1e-8) at the float32 layer's tolerance, 1e-4 of the largest gradient for every logit moved. A clipped
gradient is g c rounded once: eps / 2 of its type, and 4 roundings of float32 in c (norm, sum, ratio,
product); the norm has one."""
import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import grouped as G

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _rand(*s, dtype="bf16", std=1.0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(s) * 7 + seed)
    return (torch.randn(s, device="cuda", generator=g) * std).to(DT[dtype])


def _weights(E, H, I, r, dtype, seed=0):
    n = lambda *s, k, i: _rand(*s, dtype=dtype, std=k ** -0.5, seed=seed + i)  # noqa: E731
    return dict(w_gu=n(E, 2 * I, H, k=H, i=1), a_gu=n(E, r, H, k=H, i=2), b_gu=n(E, 2 * I, r, k=r, i=3),
                w_d=n(E, H, I, k=I, i=4), a_d=n(E, r, I, k=I, i=5), b_d=n(E, H, r, k=r, i=6))


ROUTERS = [dict(score="sigmoid", groups=4, topk_groups=2, scale=2.5),
           dict(score="softmax", renorm=False), dict(score="softmax", groups=2, group_top=1)]


@pytest.mark.parametrize("kw", ROUTERS, ids=str)
@pytest.mark.parametrize("full_ft", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_layer(kw, full_ft, bias):
    mel = _mel()
    say(f"[layer grouped] {kw} full_ft={full_ft} bias={bias}")
    T, H, I, E, k, r = 37, 64, 48, 16, 3, 4
    router = mel.GroupedRouter(E, k, **kw)
    shape = mel.Shape(T, H, I, E, k, r, "f32")
    w = _weights(E, H, I, r, "f32")
    x, dy = _rand(T, H, dtype="f32"), _rand(T, H, dtype="f32", seed=1)
    logits, b = _rand(T, E, dtype="f32", seed=2), _rand(E, dtype="f32", std=0.2) if bias else None
    layer = mel.MoELoRALayer(shape, router, full_ft=full_ft)
    layer.forward(x, logits, w, route_bias=b)
    torch.cuda.synchronize()
    ids, tw = layer.topk_ids.cpu().numpy(), layer.topk_w.cpu().numpy()
    y, y_exp = layer.y.clone(), layer.y_exp.double().cpu().numpy()
    l64 = logits.double().cpu().numpy()
    rk = dict(score=router.score, renorm=router.renorm, scale=router.scale)
    ref = G.choose(l64, k, router.score, router.groups, router.topk_groups, router.group_top,
                   None if b is None else b.cpu().numpy())
    assert (ids == ref).all()
    rw = G.weights(l64, ref, **rk)
    assert np.abs(tw - rw).max() <= 1e-5 * np.abs(rw).max()
    dx, dl, grads = layer.backward(dy, logits, w, x=x)
    torch.cuda.synchronize()
    # <dy_t, y_exp of pair (t, j)>
    rows = y_exp[layer.inv_pos.cpu().numpy()].reshape(T, k, H)
    dots = np.einsum("th,tkh->tk", dy.double().cpu().numpy(), rows)
    got = dl.double().cpu().numpy()
    exact = G.weights_backward(l64, ref, dots, **rk)
    assert np.abs(got - exact).max() <= 1e-4 * np.abs(exact).max()
    v = np.random.default_rng(1).normal(size=l64.shape)
    loss = lambda z: (G.weights(z, ref, **rk) * dots).sum()  # noqa: E731
    diff = (loss(l64 + 1e-4 * v) - loss(l64 - 1e-4 * v)) / 2e-4
    moved = np.abs(v[exact != 0]).sum()
    assert abs(diff - (got * v).sum()) <= 1e-4 * np.abs(got).max() * moved
    # chunks of tokens: the same rows bit for bit
    parts = mel.MoELoRAChunkedLayer(shape, router, 3, full_ft=full_ft)
    parts.step(x, logits, dy, w, route_bias=b)
    assert torch.equal(parts.y, y) and torch.equal(parts.d_logits, dl)
    # autograd's wrapper: the same calls
    leaf = {n: t.clone().requires_grad_(not n.startswith("w_") or full_ft) for n, t in w.items()}
    xl, ll = x.clone().requires_grad_(), logits.clone().requires_grad_()
    out = mel.MoELoRAFunction.apply(xl, ll, *(leaf[n] for n in ("w_gu", "a_gu", "b_gu", "w_d", "a_d",
                                                               "b_d")), router, k, 1.0, b)
    out.backward(dy)
    assert torch.equal(out, y) and torch.equal(xl.grad, dx) and torch.equal(ll.grad, dl)
    for n in ("a_gu", "b_gu", "a_d", "b_d"):
        assert torch.equal(leaf[n].grad, grads["d" + n])


def test_refusals():
    mel = _mel()
    shape = mel.Shape(4, 64, 32, 8, 2, 4, "bf16")
    for E, k in ((16, 2), (8, 3)):
        with pytest.raises(ValueError, match="router of"):
            mel.MoELoRALayer(shape, mel.GroupedRouter(E, k))
        with pytest.raises(ValueError, match="router of"):
            mel.MoEMXLayer(shape, mel.GroupedRouter(E, k))
    layer = mel.MoELoRALayer(shape, "softmax_topk" if "softmax_topk" in mel.ROUTER_IDS
                             else next(iter(mel.ROUTER_IDS)))
    with pytest.raises(ValueError, match="route_bias"):
        layer.forward(_rand(4, 64), _rand(4, 8, dtype="f32"), _weights(8, 64, 32, 4, "bf16"),
                      route_bias=_rand(8, dtype="f32"))


def _clipped(bufs, before, norm, max_norm):
    exact = np.sqrt(sum(float((g.double() ** 2).sum()) for g in before))
    assert abs(float(norm) - exact) <= 2.0 ** -23 * exact
    c = min(1.0, max_norm / (exact + 1e-6))
    for g, b in zip(bufs, before):
        f = torch.finfo(g.dtype)
        ref = b.double() * c
        bound = (f.eps / 2 + 4 * 2.0 ** -24) * ref.abs() + f.smallest_normal * f.eps
        assert ((g.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("full_ft,shared_I,recompute", [(False, None, True), (True, 40, False)])
def test_training_step_of_a_sublayer(dtype, full_ft, shared_I, recompute):
    """Norm, router projection, grouped routing, experts and their backward, then clipping: eagerly,
    and captured and replayed with other inputs in place."""
    mel = _mel()
    say(f"[sublayer grouped] {dtype} full_ft={full_ft} shared={shared_I}")
    T, H, I, E, k, r = 70, 64, 48, 16, 4, 8
    router = mel.GroupedRouter(E, k, groups=4, topk_groups=2, scale=1.5)
    sub = mel.MoELoRASublayer(mel.Shape(T, H, I, E, k, r, dtype), router, shared_I, post="rms",
                              full_ft=full_ft, recompute=recompute)
    w = _weights(E, H, I, r, dtype)
    sw = None
    if shared_I:
        sw = {n: t[0] for n, t in _weights(1, H, shared_I, r, dtype, seed=9).items()}
    prm = {n: 1 + _rand(*s, dtype=dtype, std=0.1) for n, s in sub.param_shapes().items()}
    h, dh2 = _rand(T, H, dtype=dtype), _rand(T, H, dtype=dtype, seed=1)
    w_r, bias = _rand(E, H, dtype=dtype, std=H ** -0.5), _rand(E, dtype="f32", std=0.1)

    def step():
        sub.step(h, dh2, prm, w_r, w, sw, route_bias=bias)

    step()
    torch.cuda.synchronize()
    bufs = sub._grad_buffers()
    assert len(bufs) == len(sub.grads) + (4 + 2 * full_ft) * (2 if shared_I else 1)
    before = [g.clone() for g in bufs]
    exact = np.sqrt(sum(float((g.double() ** 2).sum()) for g in before))
    for max_norm in (exact * 2, exact / 3):
        step()
        norm = sub.clip_grads(max_norm)
        torch.cuda.synchronize()
        _clipped(bufs, before, norm, max_norm)

    def whole():
        step()
        return sub.clip_grads(exact / 3)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm = whole()
    for i in range(3):
        h.copy_(_rand(T, H, dtype=dtype, seed=20 + i))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*bufs, norm, sub.h2)]
        whole()
        torch.cuda.synchronize()
        for a, b in zip(got, (*bufs, norm, sub.h2)):
            assert torch.equal(a, b), i

"""The residual-stream operators as a decoder layer uses them: attention's projection into the
stream, norm, MoE block (router, routed experts, shared expert), norm, gate and dropout back into
the stream, forward and backward, against the oracle stage by stage on the values each stage was
handed (so both sides route the same tokens the same way), at the layer tolerances."""
import numpy as np
import pytest
import torch

import oracle
from oracle import residual as R
from workloads import PARITY_CONFIGS, make_block_inputs
from workloads.synth import to_numpy

from gpu_util import TOL, WEIGHTS, close, say

pytestmark = pytest.mark.gpu

CASES = [  # layer, shared width, attention width, options
    ("mini-bf16", 136, 264, dict(attn_bias=True, dropout=0.2)),
    ("mini-renorm", None, None, dict(norm="layer", post="rms", alpha=0.5, weight_shift=1.0)),
    ("mini-f32", 72, 200, dict(post="layer", gate="token", gate_sigmoid=True, dropout=0.1)),
    ("mini-f16", 104, 8, dict(gate="channel", alpha=-0.5)),
    ("mini-T1", 64, 512, dict(attn_bias=True, post="rms", gate="full", dropout=0.5)),
]


def _build(name, shared_I, width, kw):
    import mixture_experts_lora_amd as mel
    cfg = PARITY_CONFIGS[name]
    inp = make_block_inputs(cfg, 5, device="cuda", shared_I=shared_I)
    sub = mel.MoELoRASublayer(mel.Shape.of(cfg), cfg.router, shared_I, attn_width=width, **kw)
    g = torch.Generator(device="cuda")
    g.manual_seed(99)
    dt = inp["x"].dtype
    new = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    prm = {}
    for n, s in sub.param_shapes().items():
        if n == "gate":
            prm[n] = new(*s).to(dt)
        elif n == "w_o":
            prm[n] = (new(*s) * s[1] ** -0.5).to(dt)
        else:
            prm[n] = (0.1 * new(*s) + (1 - kw.get("weight_shift", 0) if n[0] == "w" else 0)).to(dt)
    attn = None if width is None else new(cfg.T, width).to(dt)
    args = dict(params=prm, w_r=inp["w_r"], weights={n: inp[n] for n in WEIGHTS},
                shared_weights={n: inp["shared_" + n] for n in WEIGHTS} if shared_I else None,
                attn=attn, rng=torch.tensor([31, 1000], device="cuda"), site=6)
    return cfg, inp, sub, args


@pytest.mark.parametrize("name,shared_I,width,kw", CASES, ids=[c[0] for c in CASES])
def test_sublayer_matches_oracle(name, shared_I, width, kw):
    cfg, inp, sub, args = _build(name, shared_I, width, kw)
    say(f"[sublayer] {name} shared_I={shared_I} attn={width} {kw}")
    tol = TOL[cfg.dtype]
    h, dh2 = 2 * inp["x"], inp["dy"]
    sub.forward(h, **args)
    torch.cuda.synchronize()
    N = lambda t: to_numpy(t).astype(np.float64)  # noqa: E731
    P = {n: N(t) for n, t in args["params"].items()}
    p, eps, shift = kw.get("dropout", 0.0), 1e-5, kw.get("weight_shift", 0.0)
    norm = kw.get("norm", "rms")
    if width is not None:
        ref, _ = R.linear(N(args["attn"]), P["w_o"], P.get("b_o"), N(h), "none", (p, 31, 1000, 6))
        close("h1", to_numpy(sub.h1), ref, tol)
    h1 = N(sub.stream_in)
    close("x", to_numpy(sub.x), R.norm(h1, norm, eps, shift + P["w_pre"], P.get("b_pre")), tol)
    x = to_numpy(sub.x)
    hw = {n: to_numpy(v) for n, v in inp.items()}
    shared = {n: hw["shared_" + n] for n in WEIGHTS} if shared_I else None
    logits = to_numpy(sub.block.logits)
    close("logits", logits, oracle.router_logits(x, hw["w_r"], np.float64), 1e-5)
    after = dict(post=kw.get("post", "none"), pre="none", gate=kw.get("gate", "none"),
                 gate_sigmoid=kw.get("gate_sigmoid", False), alpha=kw.get("alpha", 1.0), eps=eps,
                 weight_shift=shift, drop=(p, 31, 1000, 7))
    y = N(sub.y)
    close("h2", to_numpy(sub.h2), R.residual_norm(h1, y, P, **after)[0], tol)
    sub.backward(dh2, **args)
    torch.cuda.synchronize()
    G = R.residual_norm_bwd(N(dh2), None, None, y, P, **after)
    close("dy", to_numpy(sub.dy), G.pop("dy"), tol)
    Y, g = oracle.layer_with_router_and_shared(x, hw["w_r"], to_numpy(sub.dy), hw, shared, cfg.k,
                                               cfg.router, cfg.lora_scale, logits=logits)
    close("y", y, Y, tol)
    dx = to_numpy(sub.block.routed.dx)
    close("dx", dx, g["dx"], tol)
    for n in ("da_gu", "db_gu", "da_d", "db_d"):
        close(n, to_numpy(sub.block.routed.grads[n]), g[n], tol)
    B = R.residual_norm_bwd(N(dh2), dx.astype(np.float64), h1, None, P, pre=norm, eps=eps,
                            weight_shift=shift)
    close("dh", to_numpy(sub.dh), B.pop("dh"), tol)
    G.pop("dh")
    G.update(B)
    if width is not None:
        _, da, G["dw_o"], G["db_o"] = R.linear_bwd(N(sub.dh), N(args["attn"]), P["w_o"], None,
                                                   "none", (p, 31, 1000, 6))
        close("dattn", to_numpy(sub.dattn), da, tol)
    assert set(sub.grads) == {"d" + n for n in P}
    for n, t in sub.grads.items():
        close(n, to_numpy(t), G[n], tol)


@pytest.mark.parametrize("name", ["mini-bf16", "mini-f32"])
def test_captured_sublayer_step_replays_like_the_eager_one(name):
    cfg, inp, sub, args = _build(*next(c for c in CASES if c[0] == name))
    say(f"[sublayer graph] {name}")
    h, dh2 = 2 * inp["x"], inp["dy"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sub.step(h, dh2, **args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dh, dattn, lora, shared = sub.step(h, dh2, **args)
    outs = [sub.h2, dh, dattn, *lora.values(), *sub.grads.values()]
    seen = []
    for offset in (4, 8, 4):
        args["rng"][1] = offset
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        sub.step(h, dh2, **args)
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b)
        seen.append(got[0])
    assert torch.equal(seen[0], seen[2]) and not torch.equal(seen[0], seen[1])


def test_sublayer_trains_only_what_it_is_told():
    import mixture_experts_lora_amd as mel
    cfg, inp, full, args = _build("mini-bf16", None, 264, dict(attn_bias=True, dropout=0.2))
    say("[sublayer train]")
    part = mel.MoELoRASublayer(mel.Shape.of(cfg), cfg.router, attn_width=264, attn_bias=True,
                               dropout=0.2, train=("w_pre",))
    a = full.step(inp["x"], inp["dy"], **args)
    b = part.step(inp["x"], inp["dy"], **args)
    torch.cuda.synchronize()
    assert set(part.grads) == {"dw_pre"} and torch.equal(part.grads["dw_pre"], full.grads["dw_pre"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("name,shared_I,opts", [
    ("mini-bf16", 136, dict(full_ft=True)), ("mini-f32", 72, dict(recompute=True)),
    ("mini-f16", 104, dict(full_ft=True, recompute=True)), ("mini-renorm", None, dict(full_ft=True)),
])
def test_sublayer_passes_the_blocks_options_and_gradients_on(name, shared_I, opts):
    """The block's own run (tested against the oracle elsewhere) on the input and output gradient
    that the sublayer handed its block: the router logits', LoRA and base gradients bit for bit."""
    import mixture_experts_lora_amd as mel
    cfg, inp, sub, args = _build(name, shared_I, 264, dict(dropout=0.1, post="rms", **opts))
    say(f"[sublayer options] {name} {opts}")
    _, _, lora, shared = sub.step(2 * inp["x"], inp["dy"], **args)
    blk = mel.MoELoRABlock(mel.Shape.of(cfg), cfg.router, shared_I, **opts)
    _, dl, lora2, shared2 = blk.step(sub.x, args["w_r"], sub.dy, args["weights"],
                                     args["shared_weights"])
    torch.cuda.synchronize()
    assert torch.equal(sub.d_logits, dl) and sub.d_logits.abs().max() > 0
    pairs = [(lora, lora2), (shared or {}, shared2 or {})]
    if opts.get("full_ft"):
        pairs.append((sub.block.routed.base_grads, blk.routed.base_grads))
        if shared_I:
            pairs.append((sub.block.shared.base_grads, blk.shared.base_grads))
    for a, b in pairs:
        assert a.keys() == b.keys()
        assert all(torch.equal(a[n], b[n]) and a[n].isfinite().all() for n in a)


def test_sublayer_run_on_its_own_output_has_no_backward():
    """Forward in place is the same numbers, but the norm's input is gone; with a projection the
    backward reads h1 instead and runs."""
    say("[sublayer in place]")
    for width in (None, 264):
        cfg, inp, sub, args = _build("mini-bf16", None, width, {})
        h = 2 * inp["x"]
        want = sub.forward(h, **args).clone()
        dh = sub.backward(inp["dy"], **args)[0].clone()
        sub.h2.copy_(h)
        assert torch.equal(sub.forward(sub.h2, **args), want)
        if width is None:
            with pytest.raises(ValueError, match="own output"):
                sub.backward(inp["dy"], **args)
        else:
            assert torch.equal(sub.backward(inp["dy"], **args)[0], dh)


def test_sublayer_projection_of_its_own_output_has_no_backward():
    say("[sublayer attn in place]")
    cfg, inp, sub, args = _build("mini-bf16", None, PARITY_CONFIGS["mini-bf16"].H, {})
    args["attn"] = sub.h2.copy_(inp["x"])
    sub.forward(2 * inp["x"], **args)
    with pytest.raises(ValueError, match="own output"):
        sub.backward(inp["dy"], **args)

"""The microscaled products where larger tiles take them, and in the ways a program may call them: in a
captured graph, on two streams at once, with rows that are nobody's, with NaN blocks and with outputs
inside larger buffers."""
import numpy as np
import pytest
import torch

from gpu_util import say
from test_gpu_mx_linear import DT, _mel, _operand, _routing, check

pytestmark = pytest.mark.gpu


# 128 or 256 rows and columns a tile: whole and cut tiles, one and several stages of 128 elements
@pytest.mark.parametrize("T,K,N,fmt,out,act", [
    (1100, 416, 3104, "fp8", "bf16", "none"), (1100, 32, 3104, "fp4", "mx8", "none"),
    (1030, 800, 1600, "fp8", "mx8", "swiglu"), (1030, 544, 1608, "fp4", "f16", "swiglu"),
    (2056, 160, 6240, "fp8", "mx8", "none"), (2056, 800, 6248, "fp4", "bf16", "none"),
    (2300, 416, 3136, "fp8", "f16", "swiglu"), (2300, 32, 3136, "fp4", "mx8", "swiglu"),
])
def test_large_tiles(T, K, N, fmt, out, act):
    check(T, K, N, fmt, out, act)


@pytest.mark.parametrize("T,K,N,E,k,skew", [
    (300, 416, 3520, 6, 3, False), (400, 160, 1984, 8, 2, True), (1500, 288, 4640, 5, 2, False),
    (1200, 544, 2624, 8, 2, True),
])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("gather", [False, True])
def test_large_tiles_of_experts(T, K, N, E, k, skew, fmt, gather):
    check(T, K, N, fmt, "bf16", "none", E, k, gather, skew=skew)
    check(T, K, N // 64 * 32, fmt, "mx8", "swiglu", E, k, gather, skew=skew)


@pytest.mark.parametrize("T,K,N,E,k", [(2300, 160, 8352, 0, 1), (2300, 416, 8360, 0, 1),
                                       (1500, 544, 6496, 5, 2)])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("out", ["bf16", "mx8"])
def test_tiles_of_192_columns(T, K, N, E, k, fmt, out):
    """Sizes whose last round of tiles of 256 columns would be mostly empty."""
    check(T, K, N // 32 * 32 if out == "mx8" else N, fmt, out, "none", E, k, gather=E > 0)


def _product(mel, T, K, N, E=0, k=1, out="bf16", act="none", gather=False, fmt="fp8", seed=0):
    """(run, y, y_scales, tensors) of a product with its own buffers."""
    rng = np.random.default_rng(seed + T + N)
    sh = mel.MXLinear(T, K, N, a_format=fmt, out=out, act=act, E=E, k=k, gather=gather)
    n_w = N * (2 if act == "swiglu" else 1)
    t = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    a, a_s, _ = _operand(rng, (T if gather else T * k, K), fmt)
    w, w_s, _ = _operand(rng, (E, n_w, K) if E else (n_w, K), "fp4", K ** -0.5)
    x = dict(a=t(a), a_s=t(a_s), w=t(w), w_s=t(w_s), rows=None, offsets=None)
    if E:
        offsets, rows = _routing(rng, T, E, k)
        x.update(offsets=t(offsets), rows=t(rows) if gather else None)
    mx = out == "mx8"
    y = torch.full((T * k, N), 7, device="cuda", dtype=torch.uint8 if mx else DT[out])
    ys = torch.full((T * k, mel.mx_scale_cols(N)), 7, device="cuda", dtype=torch.uint8) if mx else None

    def run(stream=None):
        mel.moe_mx_linear(sh, x["a"], x["a_s"], x["w"], x["w_s"], y, y_scales=ys, rows=x["rows"],
                          offsets=x["offsets"], stream=stream)

    return run, y, ys, x


CALLS = [dict(T=3, K=512, N=96, E=8, k=2, out="mx8", act="swiglu", gather=True),
         dict(T=200, K=416, N=160, E=8, k=2, gather=True),
         dict(T=1100, K=160, N=3104, out="mx8"), dict(T=2056, K=160, N=6240, fmt="fp4")]


@pytest.mark.parametrize("case", CALLS, ids=str)
def test_captured(case):
    mel = _mel()
    say(f"[mx_linear captured] {case}")
    run, y, ys, x = _product(mel, **case)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    rng = np.random.default_rng(5)
    for i in range(4):
        # other rows in the same place
        x["a"].copy_(x["a"][torch.from_numpy(rng.permutation(len(x["a"]))).cuda()])
        y.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        got, got_s = y.clone(), None if ys is None else ys.clone()
        y.fill_(7)
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, y) and (ys is None or torch.equal(got_s, ys)), i
        torch.randn(1 << 16, device="cuda").sum()


def test_two_streams():
    mel = _mel()
    say("[mx_linear streams]")
    calls = [_product(mel, seed=i, **c) for i, c in enumerate(CALLS)]
    want = []
    for run, y, _, _ in calls:
        run()
        torch.cuda.synchronize()
        want.append(y.clone())
        y.fill_(7)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, (run, _, _, _) in enumerate(calls):
            if i % 2:
                run(stream=streams[1])
            else:
                with torch.cuda.stream(streams[0]):
                    run()
    torch.cuda.synchronize()
    for (_, y, _, _), ref in zip(calls, want):
        assert torch.equal(y, ref)


@pytest.mark.parametrize("T", [4, 90, 700, 2100])
@pytest.mark.parametrize("out", ["bf16", "mx8"])
def test_rows_of_nobody(T, out):
    """Rows before offsets[0], between two experts and behind offsets[E] keep what they held."""
    mel = _mel()
    say(f"[mx_linear nobody] T={T} {out}")
    E, N = 4, 3200
    run, y, ys, x = _product(mel, T, 96, N, E=E, k=1, out=out)
    x["offsets"].copy_(torch.tensor([0, 0, T, T, T], dtype=torch.int32))
    run()
    torch.cuda.synchronize()
    whole, whole_s = y.clone(), None if ys is None else ys.clone()
    lo, hi = T // 4, T - T // 3
    x["offsets"].copy_(torch.tensor([lo, lo, hi, hi, hi], dtype=torch.int32))
    for v in (y, ys):
        if v is not None:
            v.fill_(7)
    run()
    torch.cuda.synchronize()
    for v, all_rows in ((y, whole), (ys, whole_s)):
        if v is not None:
            assert torch.equal(v[lo:hi], all_rows[lo:hi])
            assert (v[:lo] == 7).all() and (v[hi:] == 7).all()


@pytest.mark.parametrize("T,N", [(5, 64), (70, 64), (1100, 3104), (2056, 6240)])
@pytest.mark.parametrize("out", ["bf16", "mx8"])
def test_nan_blocks(T, N, out):
    """A block of scale 255 makes its row's (or its column's) results NaN and no others."""
    mel = _mel()
    say(f"[mx_linear nan] T={T} N={N} {out}")
    run, y, ys, x = _product(mel, T, 160, N, out=out)
    run()
    torch.cuda.synchronize()
    clean = y.clone()
    row, col = T - 2, N - 3
    x["a_s"][row, 2] = 255
    x["w_s"][col, 4] = 255
    run()
    torch.cuda.synchronize()
    if out == "bf16":
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[row], bad[:, col] = True, True
        assert y.isnan()[bad].all() and torch.equal(y[~bad], clean[~bad])
    else:
        assert (ys[row, :N // 32] == 255).all() and (ys[:, N // 32 - 1] == 255).all()
        keep = torch.ones_like(y, dtype=torch.bool)
        keep[row], keep[:, N - 32:] = False, False
        assert torch.equal(y[keep], clean[keep])
        ys[row, :N // 32] = 0
        assert (ys[:, :N // 32 - 1] != 255).all()


@pytest.mark.parametrize("case", CALLS, ids=str)
def test_neighbours_are_left_alone(case):
    mel = _mel()
    say(f"[mx_linear neighbours] {case}")
    run, y, ys, x = _product(mel, **case)
    T, K, N, E, k = (case.get(n, d) for n, d in (("T", 0), ("K", 0), ("N", 0), ("E", 0), ("k", 1)))
    sh = mel.MXLinear(T, K, N, a_format=case.get("fmt", "fp8"), out=case.get("out", "bf16"),
                      act=case.get("act", "none"), E=E, k=k, gather=case.get("gather", False))
    run()
    pad = 4096
    n = y.numel()
    big = torch.full((n + 2 * pad,), 7, device="cuda", dtype=y.dtype)
    inner = big[pad:pad + n].view(y.shape)
    sb = si = None
    if ys is not None:
        sb = torch.full((ys.numel() + 2 * pad,), 7, device="cuda", dtype=ys.dtype)
        si = sb[pad:pad + ys.numel()].view(ys.shape)
    mel.moe_mx_linear(sh, x["a"], x["a_s"], x["w"], x["w_s"], inner, y_scales=si, rows=x["rows"],
                      offsets=x["offsets"])
    torch.cuda.synchronize()
    assert torch.equal(inner, y)
    for v in (big, sb):
        if v is not None:
            assert (v[:pad] == 7).all() and (v[-pad:] == 7).all()


def test_refusals():
    mel = _mel()
    run, y, ys, x = _product(mel, 8, 64, 32, E=4, k=2, out="mx8", act="swiglu", gather=True)
    sh = mel.MXLinear(8, 64, 32, out="mx8", act="swiglu", E=4, k=2, gather=True)
    args = dict(a=x["a"], a_scales=x["a_s"], w=x["w"], w_scales=x["w_s"], y=y, y_scales=ys,
                rows=x["rows"], offsets=x["offsets"])

    def call(**kw):
        mel.moe_mx_linear(sh, **{**args, **kw})

    call()
    for name in args:
        with pytest.raises((TypeError, ValueError)):
            call(**{name: None})
        with pytest.raises((TypeError, ValueError)):
            call(**{name: args[name].cpu()})
        with pytest.raises((TypeError, ValueError)):
            call(**{name: args[name].float()})
        with pytest.raises((TypeError, ValueError)):
            call(**{name: args[name][1:]})
    with pytest.raises((ValueError, RuntimeError)):
        call(y=x["a"].new_empty(16, 64)[:, ::2])
    with pytest.raises(RuntimeError):
        call(y_scales=x["a_s"].new_empty(0).set_(y.untyped_storage(), 0, ys.shape, ys.stride()))
    for bad in (dict(K=48), dict(N=40), dict(k=5), dict(E=2000, k=2), dict(E=0, k=2)):
        kw = {**dict(T=8, K=64, N=32, out="mx8", act="swiglu", E=4, k=2, gather=True), **bad}
        with pytest.raises((ValueError, RuntimeError)):
            mel.moe_mx_linear_workspace_bytes(mel.MXLinear(**kw))

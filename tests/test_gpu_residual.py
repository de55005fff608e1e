"""GPU parity of dropout and the residual operator against the float64 oracle.

Tolerances. u = eps / 2 of the storage type (half a unit of rounding), e = 2^-24 that of float32.

- dropout is one float32 product rounded once: compared bit for bit with that.
- Row results (h', x', dh, dy, a token or full gate's gradient): |got - ref| <= u |ref| for the
  one rounding, plus 256 e times the largest term of the row. A row sum runs over at most 64
  elements a thread (32 e of its magnitude on average, 64 e at worst), then a tree of at most ten
  steps; an element takes two such sums, about 15 further operations, a square root and a divide:
  below 256 e of the largest term. x' is compared with the norm of the h' that the GPU stored.
- Column sums over T rows: u |ref| plus (n + 128) e sum_t |term|, n the rows of a group, the
  groups of one lane of the second pass and its 32 row sums.
"""
import numpy as np
import pytest
import torch

from oracle import residual as R

from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E = 2.0 ** -24


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _np(t):
    return t.detach().double().cpu().numpy()


def _rng(seed=77, offset=123):
    return torch.tensor([seed, offset], device="cuda", dtype=torch.int64)


def within(name, got, ref, dtype, extra):
    got, ref = _np(got), np.asarray(ref)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), name
    u = torch.finfo(DT[dtype]).eps / 2
    tiny = float(torch.finfo(DT[dtype]).smallest_normal) * torch.finfo(DT[dtype]).eps
    bound = u * np.abs(ref) * (1 + 4 * u) + extra + tiny
    diff = np.abs(got - ref)
    if not (diff <= bound).all():
        i = np.unravel_index(int(np.argmax(diff - bound)), diff.shape)
        raise AssertionError(f"{name}: {int((diff > bound).sum())} of {diff.size} outside; at {i}: "
                             f"got {got[i]:.8e} ref {ref[i]:.8e} bound {np.broadcast_to(bound, diff.shape)[i]:.2e}")


# ------------------------------------------------------------------ dropout
def _dropped(src, p, seed, offset, site):
    """The float32 product, rounded once; dropped elements are 0."""
    keep = torch.from_numpy(R.dropout_keep(src.numel(), p, seed, offset, site)).view(src.shape)
    t = R.dropout_threshold(p)
    scale = torch.tensor(65536.0 / (65536 - t), dtype=torch.float32)
    v = src.cpu().float() * scale
    return torch.where(keep, v, torch.zeros_like(v)).to(src.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 2049, 300 * 584, 1000003])
def test_dropout_is_the_mask_and_one_rounding(dtype, n):
    mel = _mel()
    say(f"[dropout] n={n} {dtype}")
    src = torch.randn(n, device="cuda").to(DT[dtype])
    for p in (0.0, 0.1, 0.5):
        dst = torch.full_like(src, 7.0)
        mel.moe_dropout(src, dst, p, _rng(), site=5)
        assert torch.equal(dst.cpu(), _dropped(src, p, 77, 123, 5)), p
    inplace = src.clone()
    mel.moe_dropout(inplace, inplace, 0.5, _rng(), site=5)
    assert torch.equal(inplace, dst)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_dropout_unaligned_and_its_neighbours(dtype):
    mel = _mel()
    say(f"[dropout unaligned] {dtype}")
    buf = torch.randn(1031, device="cuda").to(DT[dtype])
    out = torch.full((1040,), 3.0, device="cuda").to(DT[dtype])
    for so, do in ((1, 0), (0, 3), (5, 5)):
        out.fill_(3.0)
        mel.moe_dropout(buf[so:so + 1003], out[do:do + 1003], 0.3, _rng(-4, -9), site=2)
        assert torch.equal(out[do:do + 1003].cpu(), _dropped(buf[so:so + 1003], 0.3, -4, -9, 2))
        assert (out[:do] == 3).all() and (out[do + 1003:] == 3).all()


def test_dropped_infinities_are_zero_and_kept_ones_stay():
    mel = _mel()
    say("[dropout inf]")
    keep = torch.from_numpy(R.dropout_keep(512, 0.5, 77, 123))
    src = torch.full((512,), float("inf"), device="cuda", dtype=torch.bfloat16)
    src[::2] = float("nan")
    dst = torch.empty_like(src)
    mel.moe_dropout(src, dst, 0.5, _rng())
    dst, src = dst.cpu(), src.cpu()
    assert (dst[~keep] == 0).all()
    assert torch.equal(dst[keep].isnan(), src[keep].isnan())
    assert torch.equal(dst[keep].isinf(), src[keep].isinf())


def test_dropout_far_element_indexes():
    """Element indexes past 2^32: the counter's high word and 64-bit addresses."""
    mel = _mel()
    n = (1 << 32) + 8 * 5 + 3
    say(f"[dropout far] n={n}")
    src = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    mel.moe_dropout(src, src, 0.5, _rng())
    first = _dropped(torch.ones(4096, dtype=torch.bfloat16), 0.5, 77, 123, 0)
    assert torch.equal(src[:4096].cpu(), first)
    lo = (1 << 32) - 64
    ctr = np.arange(lo // 8, (n + 7) // 8, dtype=np.uint64)
    words = R.philox4x32((ctr & np.uint64(R.MASK32), ctr >> np.uint64(32), 123, 0), (77, 0))
    u16 = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1)
    want = np.where(u16.reshape(-1)[:n - lo] >= 32768, 2.0, 0.0)
    assert np.array_equal(_np(src[lo:]), want)


def test_dropout_of_more_threads_than_a_grid_holds():
    """2^35 elements are 2^32 threads, one more than a launch may have: in place, around the
    borders of the parts and at the end."""
    mel = _mel()
    n = (1 << 35) + 8 * 5 + 3
    if torch.cuda.mem_get_info()[0] < 2 * n + (8 << 30):
        pytest.skip("needs 72 GiB of free GPU memory")
    say(f"[dropout huge] n={n}")
    src = torch.ones(n, device="cuda", dtype=torch.bfloat16)
    mel.moe_dropout(src, src, 0.5, _rng())
    for lo, hi in ((0, 4096), ((1 << 34) - 64, (1 << 34) + 64), ((1 << 35) - 64, n)):
        ctr = np.arange(lo // 8, (hi + 7) // 8, dtype=np.uint64)
        words = R.philox4x32((ctr & np.uint64(R.MASK32), ctr >> np.uint64(32), 123, 0), (77, 0))
        u16 = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1)
        want = np.where(u16.reshape(-1)[:hi - lo] >= 32768, 2.0, 0.0)
        assert np.array_equal(_np(src[lo:hi]), want), lo
    del src
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ residual
# (T, H): every width class of both kernels, T odd and down to one token
SHAPES = [(1, 8), (5, 200), (333, 512), (67, 584), (129, 1024), (40, 2048), (300, 2880), (3, 4096),
          (33, 7168), (11, 8000), (2, 16384), (9, 8200)]
# (post, pre, gate, sigmoid, alpha, shift, p)
FORMS = [("none", "rms", "none", False, 1.0, 0.0, 0.0),
         ("rms", "rms", "channel", False, 0.5, 1.0, 0.1),
         ("layer", "layer", "token", True, 1.0, 0.0, 0.0),
         ("none", "layer", "full", True, 0.3, 0.0, 0.25),
         ("rms", "none", "token", False, 1.0, 1.0, 0.5),
         ("none", "none", "none", False, 1.0, 0.0, 0.3),
         ("layer", "none", "channel", True, -1.0, 0.0, 0.0),
         ("rms", "rms", "none", False, 0.22, 1.0, 0.1), ("layer", "rms", "none", False, 1.0, 0.0, 0.0),
         ("none", "layer", "none", False, 1.0, 1.0, 0.05), ("rms", "none", "full", False, 2.0, 0.0, 0.0)]


def _case(mel, T, H, dtype, form, seed=0):
    post, pre, gate, sig, alpha, shift, p = form
    d = mel.Residual(T, H, dtype, post=post, pre=pre, gate=gate, gate_sigmoid=sig, alpha=alpha,
                     weight_shift=shift, dropout=p)
    g = torch.Generator(device="cuda")
    g.manual_seed(T * 31 + H + seed)
    new = lambda *s: torch.randn(s, device="cuda", generator=g).to(DT[dtype])  # noqa: E731
    prm = {n: (0.1 * new(*s)).add(1 - shift if n[0] == "w" else 0) if n != "gate" else new(*s)
           for n, s in d.param_shapes().items()}
    return d, prm, 2 * new(T, H), new(T, H), new


def _kw(d):
    return dict(post=d.post, pre=d.pre, gate=d.gate, gate_sigmoid=d.gate_sigmoid,
                alpha=np.float32(d.alpha).astype(np.float64), eps=float(np.float32(d.eps)),
                weight_shift=d.weight_shift, drop=(d.dropout, 77, 123, 4))


def _fwd(mel, d, h, y, prm, site=4):
    T, H = d.T, d.H
    h_out = torch.full((T, H), float("nan"), device="cuda", dtype=d.torch_dtype)
    x_out = torch.full_like(h_out, float("nan")) if d.pre != "none" else None
    stats = torch.full((T, 4), float("nan"), device="cuda")
    mel.moe_residual_norm_fwd(d, h, y, prm, h_out, x_out, stats, rng=_rng(), site=site)
    return h_out, x_out, stats


def _rowmax(*terms):
    return sum(np.abs(t).max(-1, keepdims=True) for t in terms)


@pytest.mark.parametrize("form", FORMS, ids=lambda f: "-".join(str(v) for v in f[:4]))
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_residual_forward_and_backward(dtype, T, H, form):
    mel = _mel()
    say(f"[residual] {dtype} T={T} H={H} {form}")
    d, prm, h, y, new = _case(mel, T, H, dtype, form)
    kw = _kw(d)
    P = {n: _np(t) for n, t in prm.items()}
    h_out, x_out, stats = _fwd(mel, d, h, y, prm)
    ref, v, add = R.residual_norm(_np(h), _np(y), P, **kw)
    b = np.abs(P["b_post"]).max() if "b_post" in P else 0.0
    scale = _rowmax(_np(h), kw["alpha"] * add) + abs(kw["alpha"]) * b
    within("h_out", h_out, ref, dtype, 256 * E * scale)
    stored = _np(h_out)
    st = np.zeros((T, 4))
    if d.post != "none":
        st[:, 0], st[:, 1] = R.norm_stats(_np(y), d.post, kw["eps"])
    if d.pre != "none":
        st[:, 2], st[:, 3] = R.norm_stats(stored, d.pre, kw["eps"])
        w, bb = kw["weight_shift"] + P["w_pre"], P.get("b_pre")
        xr = R.norm(stored, d.pre, kw["eps"], w, bb)
        within("x_out", x_out, xr, dtype, 256 * E * _rowmax(xr, st[:, 3:] * stored * w))
    # a mean within 128 e of the row's mean magnitude, 1 / deviation within 128 e of itself
    tol = 128 * E * np.stack([np.abs(_np(y)).mean(1), st[:, 1], np.abs(stored).mean(1), st[:, 3]], 1)
    assert (np.abs(_np(stats) - st) <= tol + E * np.abs(st)).all()

    dh_out, dx_out = new(T, H), new(T, H) if d.pre != "none" else None
    dh, dy = torch.full_like(h, float("nan")), torch.full_like(h, float("nan"))
    grads = {"d" + n: torch.full_like(t, float("nan")) for n, t in prm.items()}
    ws = torch.empty(max(1, mel.moe_residual_norm_workspace_bytes(d)), device="cuda",
                     dtype=torch.uint8)
    mel.moe_residual_norm_bwd(d, dh_out, dx_out, h_out, y, prm, stats, dh, dy, grads, ws,
                              rng=_rng(), site=4)
    G = R.residual_norm_bwd(_np(dh_out), None if dx_out is None else _np(dx_out), stored, _np(y),
                            P, **kw)
    # the largest terms along a row: of D, then of everything behind the gate
    rd = _rowmax(_np(dh_out))
    if d.pre != "none":
        hat = (stored - st[:, 2:3]) * st[:, 3:]
        dd = _np(dx_out) * w
        rd = rd + st[:, 3:] * (_rowmax(dd) + _rowmax(hat) * np.abs(dd * hat).mean(1, keepdims=True))
    within("dh", dh, G["dh"], dtype, 256 * E * rd)
    gv, slope = R._gate(P.get("gate"), d.gate, d.gate_sigmoid)
    keep = R.dropout(np.ones((T, H)), *kw["drop"])
    e = np.abs(kw["alpha"] * gv * keep * G["dh"])
    etop = np.abs(kw["alpha"] * gv * keep).max(-1, keepdims=True) * rd
    yhat = None
    if d.post == "none":
        within("dy", dy, G["dy"], dtype, 256 * E * etop)
    else:
        yhat = (_np(y) - st[:, 0:1]) * st[:, 1:2]
        wp = np.abs(kw["weight_shift"] + P["w_post"])
        top = etop * wp.max()
        rdy = st[:, 1:2] * (top + _rowmax(yhat) * (top * np.abs(yhat)).mean(1, keepdims=True))
        within("dy", dy, G["dy"], dtype, 256 * E * rdy)
    groups = min(T, 4096)
    n = -(-T // groups) + groups // 32 + 32 + 128
    col = {}
    if d.pre != "none":
        col["dw_pre"], col["db_pre"] = _np(dx_out) * (np.abs(hat) + _rowmax(hat)), _np(dx_out)
    if d.post != "none":
        col["dw_post"], col["db_post"] = etop * (np.abs(yhat) + _rowmax(yhat)), etop + 0 * e
    if "gate" in P:
        term = np.abs(kw["alpha"] * keep) * (np.abs(v) + _rowmax(v) * 0.1 + b) * rd * slope
        if d.gate == "channel":
            col["dgate"] = term
        elif d.gate == "full":
            within("dgate", grads["dgate"], G["dgate"], dtype, 256 * E * _rowmax(term))
        else:
            within("dgate", grads["dgate"], G["dgate"], dtype, 256 * E * term.sum(1))
    for name, term in col.items():
        if name in G:
            within(name, grads["d" + name[1:]], G[name], dtype, n * E * np.abs(term).sum(0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_call_is_the_two_calls(dtype):
    """The norm is of the stream as stored, so the fused call equals the add followed by the norm
    of its result, bit for bit, and the fused mask is moe_dropout's."""
    mel = _mel()
    say(f"[residual split] {dtype}")
    d, prm, h, y, _ = _case(mel, 77, 584, dtype, ("none", "layer", "none", False, 1.0, 0.0, 0.3))
    h_out, x_out, stats = _fwd(mel, d, h, y, prm)
    add = mel.Residual(77, 584, dtype, pre="none", dropout=0.3)
    h2, _, _ = _fwd(mel, add, h, y, {})
    nrm = mel.Residual(77, 584, dtype, pre="layer")
    x2, st2 = torch.empty_like(h), torch.empty(77, 4, device="cuda")
    mel.moe_residual_norm_fwd(nrm, h2, None, prm, None, x2, st2)
    assert torch.equal(h_out, h2) and torch.equal(x_out, x2)
    assert torch.equal(stats, st2)
    if dtype == "f32":
        yd = torch.empty_like(y)
        mel.moe_dropout(y, yd, 0.3, _rng(), site=4)
        assert torch.equal(h2, h + yd)


def test_no_stream_no_output_and_in_place():
    mel = _mel()
    say("[residual optional]")
    form = ("rms", "rms", "channel", False, 0.5, 1.0, 0.0)
    d, prm, h, y, new = _case(mel, 50, 264, "bf16", form)
    a, xa, st = _fwd(mel, d, torch.zeros_like(h), y, prm)
    b, xb, _ = _fwd(mel, d, None, y, prm)
    assert torch.equal(a, b) and torch.equal(xa, xb)
    # in place: h_out is h, dh is dh_out
    h2, x2 = h.clone(), torch.empty_like(h)
    a, xa, st = _fwd(mel, d, h, y, prm)
    mel.moe_residual_norm_fwd(d, h2, y, prm, h2, x2, None)
    assert torch.equal(h2, a) and torch.equal(x2, xa)
    dho, dxo = new(50, 264), new(50, 264)
    dh, dy, dy2 = torch.empty_like(h), torch.empty_like(h), torch.empty_like(h)
    mel.moe_residual_norm_bwd(d, dho, dxo, a, y, prm, st, dh, dy, None, None)
    io = dho.clone()
    mel.moe_residual_norm_bwd(d, io, dxo, a, y, prm, st, io, dy2, None, None)
    assert torch.equal(io, dh) and torch.equal(dy, dy2)
    # no gradient at the stream itself, and the wanted outputs alone
    only = torch.empty_like(dy)
    mel.moe_residual_norm_bwd(d, None, dxo, a, y, prm, st, None, only, None, None)
    zero = torch.empty_like(dy)
    mel.moe_residual_norm_bwd(d, torch.zeros_like(dho), dxo, a, y, prm, st, None, zero, None, None)
    assert torch.equal(only, zero)
    ws = torch.empty(mel.moe_residual_norm_workspace_bytes(d), device="cuda", dtype=torch.uint8)
    full = {"d" + n: torch.empty_like(t) for n, t in prm.items()}
    mel.moe_residual_norm_bwd(d, dho, dxo, a, y, prm, st, dh, dy, full, ws)
    for n in full:
        one = {n: torch.empty_like(full[n])}
        mel.moe_residual_norm_bwd(d, dho, dxo, a, y, prm, st, None, None, one, ws)
        assert torch.equal(one[n], full[n]), n


def test_zero_rows_and_nan_rows_stay_in_their_rows():
    mel = _mel()
    say("[residual zero rows]")
    d, prm, h, y, new = _case(mel, 9, 2880, "bf16", ("layer", "layer", "none", False, 1.0, 0.0, 0.0))
    h[3], y[3] = 0, 0
    clean = _fwd(mel, d, h, y, prm)
    assert all(torch.isfinite(t).all() for t in clean)
    np.testing.assert_allclose(_np(clean[2])[3, 1], 1e-5 ** -0.5, rtol=1e-6)
    y2 = y.clone()
    y2[5, 17] = float("nan")
    got = _fwd(mel, d, h, y2, prm)
    rows = [r for r in range(9) if r != 5]
    for a, b in zip(clean, got):
        assert torch.equal(a[rows], b[rows])
        assert torch.isnan(b[5]).any()


def test_many_rows_repeat_bit_for_bit():
    """More rows than groups, and the same bits from two runs on different workspace contents."""
    mel = _mel()
    T, H = 20011, 136
    say(f"[residual repeat] T={T} H={H}")
    d, prm, h, y, new = _case(mel, T, H, "bf16", ("rms", "layer", "channel", True, 1.0, 0.0, 0.1))
    h_out, x_out, st = _fwd(mel, d, h, y, prm)
    dho, dxo = new(T, H), new(T, H)
    outs = []
    for fill in (0, 255):
        dh, dy = torch.empty_like(h), torch.empty_like(h)
        grads = {"d" + n: torch.empty_like(t) for n, t in prm.items()}
        ws = torch.full((mel.moe_residual_norm_workspace_bytes(d),), fill, device="cuda",
                        dtype=torch.uint8)
        mel.moe_residual_norm_bwd(d, dho, dxo, h_out, y, prm, st, dh, dy, grads, ws, rng=_rng(),
                                  site=4)
        outs.append([dh, dy, *grads.values()])
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    P = {n: _np(t) for n, t in prm.items()}
    G = R.residual_norm_bwd(_np(dho), _np(dxo), _np(h_out), _np(y), P, **_kw(d))
    hat = (_np(h_out) - _np(st)[:, 2:3]) * _np(st)[:, 3:]
    n = -(-T // 4096) + 4096 // 32 + 32 + 128
    within("dw_pre", grads["dw_pre"], G["dw_pre"], "bf16",
           n * E * np.abs(_np(dxo) * (np.abs(hat) + _rowmax(hat))).sum(0))
    within("db_pre", grads["db_pre"], G["db_pre"], "bf16", n * E * np.abs(_np(dxo)).sum(0))


def test_captured_calls_draw_new_masks_from_a_changed_rng():
    mel = _mel()
    say("[residual graph]")
    form = ("rms", "rms", "channel", False, 1.0, 0.0, 0.2)
    d, prm, h, y, new = _case(mel, 65, 512, "bf16", form)
    dho, dxo = new(65, 512), new(65, 512)
    rng = _rng()
    ws = torch.empty(mel.moe_residual_norm_workspace_bytes(d), device="cuda", dtype=torch.uint8)
    bufs = {n: torch.empty_like(h) for n in ("h_out", "x_out", "dh", "dy", "drop")}
    st = torch.empty(65, 4, device="cuda")
    grads = {"d" + n: torch.empty_like(t) for n, t in prm.items()}

    def step():
        mel.moe_residual_norm_fwd(d, h, y, prm, bufs["h_out"], bufs["x_out"], st, rng=rng)
        mel.moe_residual_norm_bwd(d, dho, dxo, bufs["h_out"], y, prm, st, bufs["dh"], bufs["dy"],
                                  grads, ws, rng=rng)
        mel.moe_dropout(y, bufs["drop"], 0.2, rng, site=1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    masks = []
    for offset in (5, 6, 5):
        rng[1] = offset
        for t in (*bufs.values(), *grads.values(), st):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*bufs.values(), *grads.values(), st)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (*bufs.values(), *grads.values(), st)):
            assert torch.equal(a, b)
        masks.append(got[4])
    assert torch.equal(masks[0], masks[2]) and not torch.equal(masks[0], masks[1])


@pytest.mark.parametrize("kind", ["channel", "token", "full"])
def test_sigmoid_gate_gradient_far_from_zero(kind):
    """float32, each element by itself: the slope keeps its accuracy where the gate is nearly open.
    A sigmoid of z is off by 2 |z| e for its exponential's argument and 5 e for the exponential, the
    sum and the reciprocal; the slope is two of them, and six products, a few positive terms' sums
    (256 e over a row, 4 e over three tokens) come on top: (4 |gate| + 16) e, and those."""
    mel = _mel()
    say(f"[gate slope] {kind}")
    T, H = (7, 56) if kind == "token" else (3, 56)
    far = np.array([-20.0, -8.0, -1.0, 0.0, 1.0, 8.0, 20.0], np.float32)
    gate = {"channel": np.tile(far, 8), "token": far, "full": np.tile(far, (T, 8))}[kind]
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    y, dh = (0.5 + torch.rand(T, H, device="cuda", generator=g) for _ in range(2))
    d = mel.Residual(T, H, "f32", pre="none", gate=kind, gate_sigmoid=True, alpha=0.5)
    ws = torch.empty(max(1, mel.moe_residual_norm_workspace_bytes(d)), device="cuda",
                     dtype=torch.uint8)
    raw = torch.from_numpy(gate).cuda()
    out = torch.full_like(raw, float("nan"))
    mel.moe_residual_norm_bwd(d, dh, None, None, y, {"gate": raw}, None, None, None,
                              {"dgate": out}, ws)
    z = gate.astype(np.float64)
    slope = 1.0 / ((1.0 + np.exp(-z)) * (1.0 + np.exp(z)))
    term = 0.5 * _np(y) * _np(dh)
    term = {"channel": term.sum(0), "token": term.sum(1), "full": term}[kind]
    bound = (4 * np.abs(z) + 16 + {"channel": 4, "token": 256, "full": 0}[kind]) * E
    rel = np.abs(_np(out) - term * slope) / (term * slope)
    assert (rel <= bound).all(), (rel / E).max()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropped_elements_ignore_their_gate(dtype, sigmoid):
    """A gate per element that is NaN or infinite where the mask drops: the forward adds nothing
    there, the backward passes nothing, and the rest of the row keeps its bits."""
    mel = _mel()
    say(f"[residual dropped gate] {dtype} {sigmoid}")
    T, H = 33, 584
    d, prm, h, y, new = _case(mel, T, H, dtype, ("rms", "layer", "full", sigmoid, 1.0, 0.0, 0.5))
    dropped = torch.from_numpy(~R.dropout_keep(T * H, 0.5, 77, 123, 4)).view(T, H).cuda()
    dho, dxo, gate = new(T, H), new(T, H), prm["gate"]
    runs = []
    for fill in (0.0, float("nan"), float("inf"), -float("inf")):
        prm["gate"] = torch.where(dropped, torch.full_like(gate, fill), gate)
        h_out, x_out, st = _fwd(mel, d, h, y, prm)
        dh, dy = torch.full_like(h, float("nan")), torch.full_like(h, float("nan"))
        grads = {"d" + n: torch.full_like(t, float("nan")) for n, t in prm.items()}
        ws = torch.empty(mel.moe_residual_norm_workspace_bytes(d), device="cuda", dtype=torch.uint8)
        mel.moe_residual_norm_bwd(d, dho, dxo, h_out, y, prm, st, dh, dy, grads, ws, rng=_rng(), site=4)
        assert (grads["dgate"][dropped] == 0).all() and torch.equal(h_out[dropped], h[dropped])
        runs.append([h_out, x_out, dh, dy, *grads.values()])
    for out in runs:
        assert all(torch.equal(a, c) and a.isfinite().all() for a, c in zip(runs[0], out))

"""GPU parity of the linear operator against the float64 oracle.

Tolerances. u = eps / 2 of the storage type, e = 2^-24. A float32 dot product of n terms is off by a
random walk of n roundings, each at most e of a partial sum, so by 4 sqrt(n) e sum |terms| at far
more than the walk's deviation; the epilogue adds at most 32 e of its terms (an activation's slope
is below 1.13), and the output one rounding of u. dz feeds the products rounded to the storage
type: the oracle rounds its float64 dz the same way, and where float32 and float64 fall on two
sides of a rounding border (a share of about 8 e / 2u of the elements, below one in a row of these
widths) a term differs by 2u |dz w|; eight such are allowed for.
"""
import numpy as np
import pytest
import torch

from oracle import residual as R

from gpu_util import say
from test_gpu_residual import DT, E, _np, _rng, within

pytestmark = pytest.mark.gpu

# every path: up to 1, 2, 4, 8 and 16 tokens, small tiles with slices, one slice, 256-wide tiles
SHAPES = [(1, 264, 584), (1, 8, 8), (2, 584, 264), (3, 4096, 136), (7, 1032, 264), (8, 2880, 72),
          (13, 136, 1032), (16, 264, 264), (17, 584, 264), (64, 8, 264), (129, 1032, 8),
          (300, 584, 1032), (700, 2880, 200), (1500, 72, 1032)]
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _inputs(T, K, N, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(T * 131 + K * 7 + N + seed)
    new = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    dt = DT[dtype]
    return (new(T, K).to(dt), (new(N, K) * K ** -0.5).to(dt), (0.3 * new(N)).to(dt),
            new(T, N).to(dt), new(T, N).to(dt))


def _ws(n):
    return torch.full((max(1, n),), 255, device="cuda", dtype=torch.uint8)  # NaN as float32


def _nan(*s, dtype):
    return torch.full(s, float("nan"), device="cuda", dtype=DT[dtype])


def check_fwd(mel, T, K, N, dtype, act, p, use_bias=True, use_res=True, keep_pre=True):
    x, w, b, res, _ = _inputs(T, K, N, dtype)
    b, res = b if use_bias else None, res if use_res else None
    sh = mel.LinearShape(T, K, N, dtype, act=act, dropout=p)
    y = _nan(T, N, dtype=dtype)
    pre = _nan(T, N, dtype=dtype) if keep_pre else None
    mel.moe_linear_fwd(sh, x, w, y, _ws(mel.moe_linear_workspace_bytes(sh)[0]), bias=b,
                       residual=res, pre=pre, rng=_rng(), site=4)
    drop = (p, 77, 123, 4)
    xs, ws, bs = _np(x), _np(w), _np(b) if use_bias else 0.0
    ref, z = R.linear(xs, ws, bs, _np(res) if use_res else None, act, drop)
    zerr = 4 * np.sqrt(K) * E * (np.abs(xs) @ np.abs(ws).T) + E * (np.abs(bs) + np.abs(z))
    if keep_pre:
        within("pre", pre, z, dtype, zerr)
    keep = R.dropout(np.ones((T, N)), *drop)
    extra = keep * (1.13 * zerr + 32 * E * (np.abs(z) + 1)) + 2 * E * np.abs(ref)
    within("y", y, ref, dtype, extra + (E * np.abs(_np(res)) if use_res else 0.0))
    return y


def check_bwd(mel, T, K, N, dtype, act, p):
    x, w, b, _, dy = _inputs(T, K, N, dtype)
    sh = mel.LinearShape(T, K, N, dtype, act=act, dropout=p)
    xs, ws = _np(x), _np(w)
    pre = torch.from_numpy(xs @ ws.T + _np(b)).to(DT[dtype]).cuda()
    out = {"dx": _nan(T, K, dtype=dtype), "dw": _nan(N, K, dtype=dtype), "db": _nan(N, dtype=dtype)}
    mel.moe_linear_bwd(sh, dy, x, w, pre if act != "none" else None, out["dx"], out["dw"],
                       out["db"], _ws(mel.moe_linear_workspace_bytes(sh)[1]), rng=_rng(), site=4)
    dz = R.linear_bwd(_np(dy), xs, ws, _np(pre), act, (p, 77, 123, 4))[0]
    db = dz.sum(0)
    u = torch.finfo(DT[dtype]).eps / 2
    form = act != "none" or p > 0
    dzr = _np(torch.from_numpy(dz).to(DT[dtype])) if form else dz
    # dz itself: its slope, mask and product in float32 (48 e of |dy| times the scale of the kept)
    dzerr = 48 * E * np.abs(R.dropout(_np(dy), p, 77, 123, 4)) if form else 0 * dz
    flips = 16 * u if form and dtype != "f32" else 0.0
    a, c = np.abs(dzr), dzerr.max()
    within("dx", out["dx"], dzr @ ws, dtype,
           4 * np.sqrt(N) * E * (a @ np.abs(ws)) + flips * a.max() * np.abs(ws).max() +
           (4 * np.sqrt(N) * c * np.abs(ws).max() if form else 0))
    within("dw", out["dw"], dzr.T @ xs, dtype,
           4 * np.sqrt(T) * E * (a.T @ np.abs(xs)) + flips * a.max() * np.abs(xs).max() +
           (4 * np.sqrt(T) * c * np.abs(xs).max() if form else 0))
    within("db", out["db"], db, dtype, (4 * np.sqrt(T) + 32) * E * np.abs(dz).sum(0) + T * c)
    return out


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_linear_forward(dtype, T, K, N):
    mel = _mel()
    say(f"[linear fwd] {dtype} T={T} K={K} N={N}")
    for i, act in enumerate(ACTS):
        check_fwd(mel, T, K, N, dtype, act, 0.25 if i % 2 else 0.0)
    check_fwd(mel, T, K, N, dtype, "none", 0.5, use_bias=False, keep_pre=False)
    check_fwd(mel, T, K, N, dtype, "silu", 0.0, use_bias=False, use_res=False, keep_pre=False)


@pytest.mark.parametrize("T,K,N", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_linear_backward(dtype, T, K, N):
    mel = _mel()
    say(f"[linear bwd] {dtype} T={T} K={K} N={N}")
    for i, act in enumerate(ACTS):
        check_bwd(mel, T, K, N, dtype, act, 0.0 if i % 2 else 0.25)
    check_bwd(mel, T, K, N, dtype, "none", 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,K,N", [(4000, 264, 3400), (4111, 1160, 520), (4352, 72, 4104),
                                   (4352, 4104, 72), (300, 2400, 2568), (3000, 136, 136),
                                   (4000, 3400, 264)])
def test_linear_large_tiles(dtype, T, K, N):
    """Enough tiles for the widest ones: 256 x 256 in the forward (first), 256 x 192 in the forward
    (third) and the input gradient (fourth), 192 x 192 in the weight gradient (fifth); the sixth
    splits the weight gradient's rows into many slices; 256 x 256 in the input gradient (last)."""
    mel = _mel()
    say(f"[linear large] {dtype} T={T} K={K} N={N}")
    check_fwd(mel, T, K, N, dtype, "gelu_tanh", 0.1)
    check_bwd(mel, T, K, N, dtype, "none", 0.0)


def test_linear_optional_outputs_and_in_place():
    mel = _mel()
    for T in (5, 300):
        say(f"[linear optional] T={T}")
        K, N = 264, 520
        x, w, b, res, dy = _inputs(T, K, N, "bf16")
        sh = mel.LinearShape(T, K, N, "bf16", act="gelu", dropout=0.1)
        f, bw = mel.moe_linear_workspace_bytes(sh)
        y, pre = torch.empty_like(res), torch.empty_like(res)
        mel.moe_linear_fwd(sh, x, w, y, _ws(f), bias=b, residual=res, pre=pre, rng=_rng())
        io = res.clone()
        mel.moe_linear_fwd(sh, x, w, io, _ws(f), bias=b, residual=io, rng=_rng())
        assert torch.equal(io, y)
        full = [torch.empty_like(t) for t in (x, w, b)]
        mel.moe_linear_bwd(sh, dy, x, w, pre, *full, _ws(bw), rng=_rng())
        for i in range(3):
            one = [None] * 3
            one[i] = torch.empty_like(full[i])
            mel.moe_linear_bwd(sh, dy, x if i == 1 else None, w if i == 0 else None, pre, *one,
                               _ws(bw), rng=_rng())
            assert torch.equal(one[i], full[i]), i


@pytest.mark.parametrize("T", [4, 333, 4000])
def test_linear_repeats_and_replays_bit_for_bit(T):
    mel = _mel()
    say(f"[linear graph] T={T}")
    K, N = 520, 3400 if T == 4000 else 264
    x, w, b, res, dy = _inputs(T, K, N, "bf16")
    sh = mel.LinearShape(T, K, N, "bf16", act="silu", dropout=0.2)
    f, bw = (_ws(n) for n in mel.moe_linear_workspace_bytes(sh))
    y, pre = torch.empty_like(res), torch.empty_like(res)
    out = [torch.empty_like(t) for t in (x, w, b)]
    rng = _rng()

    def step():
        mel.moe_linear_fwd(sh, x, w, y, f, bias=b, residual=res, pre=pre, rng=rng)
        mel.moe_linear_bwd(sh, dy, x, w, pre, *out, bw, rng=rng)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for offset in (1, 2, 3):
        rng[1] = offset
        for t in (y, pre, *out):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, pre, *out)]
        step()
        torch.cuda.synchronize()
        for a, c in zip(got, (y, pre, *out)):
            assert torch.equal(a, c)


def test_linear_nonfinite_inputs_stay_in_their_rows():
    mel = _mel()
    say("[linear nan]")
    for T in (6, 200):
        x, w, b, res, _ = _inputs(T, 264, 136, "bf16")
        sh = mel.LinearShape(T, 264, 136, "bf16", act="gelu")
        ws = _ws(mel.moe_linear_workspace_bytes(sh)[0])
        y0, y1 = torch.empty_like(res), torch.empty_like(res)
        mel.moe_linear_fwd(sh, x, w, y0, ws, bias=b, residual=res)
        x[2, 5] = float("nan")
        x[4, 7] = float("inf")
        mel.moe_linear_fwd(sh, x, w, y1, ws, bias=b, residual=res)
        rows = [r for r in range(T) if r not in (2, 4)]
        assert torch.equal(y0[rows], y1[rows])
        assert torch.isnan(y1[2]).all() and not torch.isfinite(y1[4]).all()


def test_float32_gelu_keeps_its_accuracy_in_the_tail():
    """z = x w^T of one term is exact, so y is gelu(z) alone and dx its slope. Phi by erfc: its
    argument is off by 2 e of it (a product and a constant), which erfc's logarithm takes times at most
    2 x^2 + 1 = z^2 + 1 for negative z: (2 z^2 + 2) e, and 12 e for erfc itself and two products. The
    density's exponential: z^2 / 2 with three roundings, (1.5 z^2) e, and 10 e for it and its products."""
    from scipy.special import erfc
    mel = _mel()
    say("[gelu f32]")
    z = np.linspace(-9, 9, 4099).astype(np.float32)
    T, n = z.size, 8
    x = torch.zeros(T, n, device="cuda")
    x[:, 0] = torch.from_numpy(z)
    w = torch.zeros(n, n, device="cuda")
    w[0, 0] = 1.0
    z = z.astype(np.float64)
    phi, pdf = 0.5 * erfc(-z * np.sqrt(0.5)), np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    eval_, edf = (2 * z * z + 14) * E * phi, (1.5 * z * z + 10) * E * np.abs(z) * pdf
    for rows in (slice(None), slice(1600, 1601), slice(1600, 1613)):
        t = x[rows].contiguous()
        sh = mel.LinearShape(t.shape[0], n, n, "f32", act="gelu")
        f, b = (_ws(m) for m in mel.moe_linear_workspace_bytes(sh))
        y = _nan(t.shape[0], n, dtype="f32")
        mel.moe_linear_fwd(sh, t, w, y, f)
        d = np.abs(_np(y)[:, 0] - (z * phi)[rows])
        assert (d <= (np.abs(z) * eval_)[rows] + 1e-38).all(), d.max()
        dx, pre = _nan(t.shape[0], n, dtype="f32"), t.clone()
        mel.moe_linear_bwd(sh, torch.ones_like(t), t, w, pre, dx, None, None, b)
        d = np.abs(_np(dx)[:, 0] - (phi + z * pdf)[rows])
        assert (d <= (eval_ + edf + E * np.abs(phi + z * pdf))[rows]).all(), d.max()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_slopes_of_huge_products_are_their_limits(act, dtype):
    """Where z^2 or z^3 overflows, and at infinity: 1 for positive z, 0 for negative, no NaN from a
    product of infinity and zero. A NaN stays one."""
    mel = _mel()
    say(f"[slope limits] {act} {dtype}")
    big = [200.0, 6e4] if dtype == "f16" else [200.0, 6e4, 1e13, 1e20, 3e38]
    z = torch.tensor([v * s for v in big + [float("inf")] for s in (1, -1)] + [float("nan")])
    T, n = z.numel(), 8
    pre = z[:, None].expand(T, n).to(DT[dtype]).cuda().contiguous()
    w = torch.eye(n, device="cuda", dtype=DT[dtype])
    dy, dx = torch.full_like(pre, 3.0), torch.empty_like(pre)
    sh = mel.LinearShape(T, n, n, dtype, act=act)
    mel.moe_linear_bwd(sh, dy, None, w, pre, dx, None, None, _ws(mel.moe_linear_workspace_bytes(sh)[1]))
    want = torch.tensor([3.0, 0.0] * (len(big) + 1))[:, None].expand(T - 1, n)
    assert torch.equal(dx[:-1].float().cpu(), want)
    assert act == "relu" or dx[-1].isnan().all()


@pytest.mark.parametrize("dtype,T", [("bf16", 530000), ("f32", 270000)])
def test_linear_operands_past_two_gigabytes(dtype, T):
    """x, y, dy and dx of 2.2e9 bytes each: rows at both ends and around byte 2^31, and a weight
    gradient whose rows have to be sliced where a tile addresses them by 32-bit offsets (bf16)."""
    mel = _mel()
    K = N = 2056
    say(f"[linear far] {dtype} T={T}")
    x, w, b, _, dy = _inputs(T, K, N, dtype)
    sh = mel.LinearShape(T, K, N, dtype)
    f, bw = (_ws(n) for n in mel.moe_linear_workspace_bytes(sh))
    y, dx, dw, db = _nan(T, N, dtype=dtype), _nan(T, K, dtype=dtype), torch.empty_like(w), torch.empty_like(b)
    mel.moe_linear_fwd(sh, x, w, y, f, bias=b)
    mel.moe_linear_bwd(sh, dy, x, w, None, dx, dw, db, bw)
    assert y.isfinite().all() and dx.isfinite().all()
    mid = (1 << 31) // (K * x.element_size())
    rows = torch.tensor([0, 1, 255, 256, mid - 1, mid, mid + 1, T // 2, T - 2, T - 1], device="cuda")
    for got, a, m, add in ((y, x, w.t(), b), (dx, dy, w, None)):
        a, m = _np(a[rows]), _np(m)
        ref = a @ m + (0 if add is None else _np(add))
        mag = np.abs(a) @ np.abs(m) + (0 if add is None else np.abs(_np(add)))
        within("rows", got[rows], ref, dtype, 4 * np.sqrt(K) * E * mag)
    cols = [0, 100, 1023, N - 1]
    d, xx = dy[:, cols].double().t().contiguous(), x.double()
    within("dw", dw[cols], _np(d @ xx), dtype, 4 * np.sqrt(T) * E * _np(d.abs() @ xx.abs_()))
    within("db", db[cols], _np(d.sum(1)), dtype, (4 * np.sqrt(T) + 32) * E * _np(d.abs().sum(1)))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,K,N", [(7, 1032, 264), (300, 584, 1032), (3000, 136, 136),
                                   (4111, 1160, 520), (4352, 4104, 72), (4000, 264, 3400)])
def test_dropout_alone_adds_no_rounding_to_the_backward(dtype, T, K, N):
    """Without an activation dz is dy or 0, and the kept elements' scale multiplies float32 sums:
    the results are off by their own sums' rounding and one of the output."""
    mel = _mel()
    say(f"[linear bwd dropout] {dtype} T={T} K={K} N={N}")
    x, w, b, _, dy = _inputs(T, K, N, dtype)
    sh = mel.LinearShape(T, K, N, dtype, dropout=0.3)
    dx, dw, db = _nan(T, K, dtype=dtype), _nan(N, K, dtype=dtype), _nan(N, dtype=dtype)
    mel.moe_linear_bwd(sh, dy, x, w, None, dx, dw, db, _ws(mel.moe_linear_workspace_bytes(sh)[1]),
                       rng=_rng(), site=4)
    xs, ws = _np(x), _np(w)
    dz, rx, rw, rb = R.linear_bwd(_np(dy), xs, ws, None, "none", (0.3, 77, 123, 4))
    a = np.abs(dz)
    for name, got, ref, n, mag in (("dx", dx, rx, N, a @ np.abs(ws)), ("dw", dw, rw, T, a.T @ np.abs(xs)),
                                   ("db", db, rb, T, a.sum(0))):
        within(name, got, ref, dtype, (4 * np.sqrt(n) * mag + 4 * np.abs(ref)) * E)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
def test_dropped_products_pass_no_gradient_whatever_they_hold(act):
    mel = _mel()
    say(f"[linear dropped nan] {act}")
    T, K, N = 65, 72, 136
    x, w, b, _, dy = _inputs(T, K, N, "bf16")
    sh = mel.LinearShape(T, K, N, act=act, dropout=0.5)
    dropped = torch.from_numpy(~R.dropout_keep(T * N, 0.5, 77, 123, 4)).view(T, N).cuda()
    pre = torch.where(dropped, torch.zeros_like(dy), dy.roll(1, 0))
    runs = []
    for fill in (0.0, float("nan"), float("inf"), -float("inf")):
        z = torch.where(dropped, torch.full_like(pre, fill), pre)
        g = torch.where(dropped, torch.full_like(dy, fill), dy)
        out = [_nan(*t.shape, dtype="bf16") for t in (x, w, b)]
        mel.moe_linear_bwd(sh, g, x, w, z, *out, _ws(mel.moe_linear_workspace_bytes(sh)[1]),
                           rng=_rng(), site=4)
        runs.append(out)
    for out in runs:
        assert all(torch.equal(a, c) and a.isfinite().all() for a, c in zip(runs[0], out))

"""GPU parity of the microscaled products against float64 products of the dequantised operands.

Tolerances. The products of two codes with their scales are exact. The matrix cores add them eight
neighbours at a time, aligned to the largest of the eight: what of a product lies below 2^-13 of the
power of two at or under that largest is cut off towards zero (measured; 256 beside 1.75 * 2^-5 gives
2^-5, and 2^-6 nothing, at the places 0 to 7 and no further). So a product's error is at most the sum
of what is cut, |a w| mod that unit, which `cut` forms product by product, and that of the float32 sums
of the eights, for which 2^-16 sum_k |a w| is allowed: d is the sum of the two. With SwiGLU, d comes in through both factors, the slope of
silu is at most 1.1, and its exponential and reciprocal add 16 roundings of float32. A 16-bit result
is rounded once: u = eps / 2 of the type. An 8-bit result is the code of some value within d of the
exact one, under the scale of some largest magnitude within d: both are checked as intervals.
"""
import numpy as np
import pytest
import torch

from oracle import microscale as X

from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
E24 = 2.0 ** -24


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _operand(rng, shape, fmt, std=1.0):
    x = rng.normal(size=shape) * std * np.exp2(rng.integers(-2, 3, size=(*shape[:-1], 1)))
    codes, scales = X.quantize(x.reshape(-1, shape[-1]), fmt)
    val = X.dequantize(codes, scales, fmt).reshape(shape)
    stored = X.pack(codes, fmt).reshape(*shape[:-1], -1)
    return stored, scales.reshape(*shape[:-1], -1), val


def _routing(rng, T, E, k, skew=False):
    """(offsets, sorted_pair) of k distinct experts a token; skew: half of the experts get none."""
    n = max(k, E // 2) if skew else E
    ids = np.stack([rng.permutation(n)[:k] for _ in range(T)])
    order = np.argsort(ids.reshape(-1), kind="stable")
    counts = np.bincount(ids.reshape(-1), minlength=E)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), order.astype(np.int32)


def cut(a, w):
    """[M, n] sums over k of what the alignment of eight products cuts off."""
    a, w = (torch.from_numpy(np.ascontiguousarray(v)).cuda().view(len(v), -1, 8) for v in (a, w))
    out = torch.zeros(len(a), len(w), device="cuda", dtype=torch.float64)
    step = max(1, (1 << 25) // w.numel())
    for lo in range(0, len(a), step):
        p = (a[lo:lo + step, None] * w[None]).abs()
        # frexp's mantissa is in [0.5, 1)
        unit = torch.exp2(torch.frexp(p.amax(-1))[1].double() - 14)[..., None]
        out[lo:lo + step] = (p - (p / unit).floor() * unit).sum((-1, -2))
    return out.cpu().numpy()


def reference(a, w, offsets, M, swiglu):
    """(y, d) in float64 for rows in expert order (offsets None: one matrix)."""
    spans = [(0, M, w)] if offsets is None else [
        (offsets[e], offsets[e + 1], w[e]) for e in range(len(offsets) - 1)]
    n_w = w.shape[-2]
    z, d = np.zeros((M, n_w)), np.zeros((M, n_w))
    for lo, hi, we in spans:
        z[lo:hi] = a[lo:hi] @ we.T
        if hi > lo:
            d[lo:hi] = 2.0 ** -16 * (np.abs(a[lo:hi]) @ np.abs(we).T) + cut(a[lo:hi], we)
    if not swiglu:
        return z, d
    n = n_w // 2
    g, u = z[:, :n], z[:, n:]
    silu = g / (1 + np.exp(-g))
    y = silu * u
    return y, 1.1 * d[:, :n] * np.abs(u) + (np.abs(silu) + d[:, :n]) * d[:, n:] + 16 * E24 * np.abs(y)


def compare(out, y, y_scales, ref, d):
    if out != "mx8":
        u = torch.finfo(DT[out]).eps / 2
        tiny = float(torch.finfo(DT[out]).smallest_normal)
        got = y.double().cpu().numpy()
        assert np.isfinite(got).all()
        bad = np.abs(got - ref) > u * np.abs(ref) + (1 + u) * d + tiny
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.abs(got - ref).max())
        return
    codes, scales = y.cpu().numpy(), y_scales.cpu().numpy()
    M, N = codes.shape
    assert (scales[:, N // 32:] == 0).all()
    s = scales[:, :N // 32].astype(np.float64)
    blocks = np.abs(ref).reshape(M, -1, 32)
    db = d.reshape(M, -1, 32)
    lo, hi = np.maximum(blocks - db, 0).max(2), (blocks + db).max(2)
    exp = lambda v: np.maximum(np.where(v > 0, np.frexp(v)[1] - 1 + 127 - 8, 0), 0)  # noqa: E731
    assert ((s >= exp(lo)) & (s <= exp(hi))).all()
    m = np.exp2(127 - s)[..., None]
    low = X.rounded((ref - d).reshape(M, -1, 32) * m, "fp8").reshape(M, N)
    high = X.rounded((ref + d).reshape(M, -1, 32) * m, "fp8").reshape(M, N)
    got = X.dequantize(codes, np.full_like(scales, 127), "fp8")
    assert ((got >= low) & (got <= high)).all()


def check(T, K, N, fmt, out, act="none", E=0, k=1, gather=False, seed=0, skew=False):
    mel = _mel()
    say(f"[mx_linear] T={T} K={K} N={N} {fmt} {out} {act} E={E} k={k} gather={gather}")
    rng = np.random.default_rng(seed + T + K + N + E)
    sh = mel.MXLinear(T, K, N, a_format=fmt, out=out, act=act, E=E, k=k, gather=gather)
    M, n_w = T * k, N * (2 if act == "swiglu" else 1)
    a, a_s, av = _operand(rng, (T if gather else M, K), fmt)
    w, w_s, wv = _operand(rng, ((E, n_w, K) if E else (n_w, K)), "fp4", K ** -0.5)
    offsets = rows = None
    if E:
        offsets, rows = _routing(rng, T, E, k, skew)
        if gather:
            av = av[rows // k]
    t = lambda v: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    mx = out == "mx8"
    y = torch.full((M, N), 7, device="cuda", dtype=torch.uint8 if mx else DT[out])
    ys = torch.full((M, mel.mx_scale_cols(N)), 7, device="cuda", dtype=torch.uint8) if mx else None
    ws = torch.empty(max(1, mel.moe_mx_linear_workspace_bytes(sh)), device="cuda", dtype=torch.uint8)
    args = (sh, t(a), t(a_s), t(w), t(w_s), y, ws)
    kw = dict(y_scales=ys, rows=t(rows) if gather else None, offsets=t(offsets))
    mel.moe_mx_linear(*args, **kw)
    torch.cuda.synchronize()
    compare(out, y, ys, *reference(av, wv, offsets, M, act == "swiglu"))
    first = y.clone()
    y.zero_()
    mel.moe_mx_linear(*args, **kw)
    assert torch.equal(first, y)


DENSE = [(1, 32, 32), (1, 2880, 320), (3, 96, 64), (16, 160, 96), (17, 512, 288), (33, 544, 32),
         (64, 1056, 512), (128, 128, 256), (129, 2880, 544), (300, 608, 288), (257, 4096, 96)]


@pytest.mark.parametrize("T,K,N", DENSE)
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("out", ["bf16", "f16", "mx8"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_one_matrix(T, K, N, fmt, out, act):
    check(T, K, N, fmt, out, act)


@pytest.mark.parametrize("N", [8, 16, 24, 40, 136, 264, 1000])
@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_odd_widths(T, N, act):
    check(T, 224, N, "fp8", "bf16", act)
    check(T, 224, N, "fp4", "f16", act)


EXPERTS = [  # T, K, N, E, k, skew
    (1, 2880, 96, 32, 4, False), (1, 64, 64, 3, 3, False), (7, 256, 128, 8, 2, True),
    (40, 512, 96, 100, 4, False), (300, 608, 192, 6, 3, False), (200, 160, 160, 130, 8, True),
    (1000, 288, 320, 4, 2, True), (64, 96, 64, 1, 1, False), (333, 416, 64, 70, 1, False),
    (90, 64, 32, 1024, 32, False),
]


@pytest.mark.parametrize("T,K,N,E,k,skew", EXPERTS)
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("gather", [False, True])
def test_experts(T, K, N, E, k, skew, fmt, gather):
    check(T, K, N, fmt, "bf16", "none", E, k, gather, skew=skew)
    check(T, K, N, fmt, "mx8", "swiglu", E, k, gather, skew=skew)

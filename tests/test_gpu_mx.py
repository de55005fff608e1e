"""GPU parity of the microscaled conversions and of the norm with an 8-bit output.

The conversions are exact functions of their input: codes, scales and values are compared bit for
bit with the float64 oracle. The norm's 8-bit rows are compared bit for bit with moe_mx_quantize of
the rows that moe_residual_norm_fwd gives."""
import numpy as np
import pytest
import torch

from oracle import microscale as X

from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _blank(mel, rows, cols, fmt):
    return (torch.full((rows, cols // 2 if fmt == "fp4" else cols), 0xAB, device="cuda", dtype=torch.uint8),
            torch.full((rows, mel.mx_scale_cols(cols)), 0xCD, device="cuda", dtype=torch.uint8))


def _check(x, fmt):
    mel = _mel()
    rows, cols = x.shape
    codes, scales = _blank(mel, rows, cols, fmt)
    mel.moe_mx_quantize(x, codes, scales, fmt)
    src = x.double().cpu().numpy()
    want, want_s = X.quantize(src, fmt)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    got = X.unpack(codes.cpu().numpy(), fmt)
    bad = (want_s[:, :cols // 32] == 255).repeat(32, 1)  # a NaN block's codes are of no account
    same = (got == want) | bad
    # the sign of a zero is of no account either
    n = 8 if fmt == "fp4" else 128
    assert (same | ((got % n == 0) & (want % n == 0))).all()
    back = torch.full_like(x, 7.0)
    mel.moe_mx_dequantize(codes, scales, back, fmt)
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(X.dequantize(want, want_s, fmt)).to(x.dtype)
    assert torch.equal(back.cpu().nan_to_num(nan=123.0, posinf=1e4, neginf=-1e4),
                       ref.nan_to_num(nan=123.0, posinf=1e4, neginf=-1e4))


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (5, 512), (7, 544), (300, 608), (33, 2880),
                                       (2, 16384), (1000, 96)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_conversions(rows, cols, dtype, fmt):
    say(f"[mx] {rows}x{cols} {dtype} {fmt}")
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * cols)
    x = torch.randn(rows, cols, device="cuda", generator=g)
    x = x * torch.randn(rows, 1, device="cuda", generator=g).mul(3).exp()
    _check(x.to(DT[dtype]), fmt)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_every_exponent_and_midpoint(fmt, dtype):
    """Blocks of every scale the type reaches, with all codes and all midpoints between them;
    zeros, the smallest subnormals, the largest values, infinities and NaN."""
    say(f"[mx exponents] {dtype} {fmt}")
    t = X.TABLE[fmt]
    vals = np.concatenate([t, (t[1:] + t[:-1]) / 2, [t[-1] * 1.1, 2.0 ** (X.TOP[fmt] + 1) * (1 - 2.0 ** -8)]])
    vals = np.concatenate([vals, -vals])
    vals = np.concatenate([vals, np.zeros(-len(vals) % 31)]).reshape(-1, 31)
    base = np.concatenate([vals, np.full((len(vals), 1), 2.0 ** X.TOP[fmt])], 1)
    lo, hi = {"f16": (-26, 7), "bf16": (-140, 119), "f32": (-150, 119)}[dtype]
    rows = [base * 2.0 ** e for e in range(lo, hi)]
    x = np.concatenate(rows).astype(np.float64)
    x = torch.from_numpy(x).to(DT[dtype]).cuda()
    extra = torch.zeros(8, 32, device="cuda", dtype=DT[dtype])
    extra[1, 3], extra[2, 31], extra[3, 0] = float("inf"), float("nan"), -float("inf")
    extra[4] = torch.finfo(DT[dtype]).max
    extra[5, 1] = torch.finfo(DT[dtype]).smallest_normal
    extra[6, 1] = -torch.finfo(DT[dtype]).smallest_normal * torch.finfo(DT[dtype]).eps
    extra[7] = -0.0
    _check(torch.cat([x, extra]).contiguous(), fmt)


def test_dequantise_every_code():
    """Every code under every scale, NaN codes and the NaN scale among them."""
    mel = _mel()
    say("[mx decode]")
    for fmt, n in (("fp4", 16), ("fp8", 256)):
        codes = np.tile(np.arange(n, dtype=np.uint8), (256, 1))
        if n == 16:
            codes = np.concatenate([codes, codes], 1)
        cols = codes.shape[1]
        scales = np.zeros((256, X.scale_cols(cols)), np.uint8)
        scales[:, :cols // 32] = np.arange(256, dtype=np.uint8)[:, None]
        out = torch.empty(256, cols, device="cuda")
        mel.moe_mx_dequantize(torch.from_numpy(X.pack(codes, fmt)).cuda(),
                              torch.from_numpy(scales).cuda(), out, fmt)
        ref = X.dequantize(codes, scales, fmt)
        with np.errstate(over="ignore"):
            assert np.array_equal(out.cpu().numpy(), ref.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("T,H", [(1, 32), (3, 2880), (37, 512), (300, 608), (64, 1056), (9, 7168),
                                 (5, 8192), (3, 8224), (2, 16384), (4100, 96)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_norm_in_8_bits(T, H, dtype):
    mel = _mel()
    say(f"[norm mx] {T}x{H} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)
    new = lambda *s: torch.randn(s, device="cuda", generator=g).to(DT[dtype])  # noqa: E731
    rng = torch.tensor([5, 6], device="cuda", dtype=torch.int64)
    for kw in (dict(), dict(post="rms", alpha=0.5, weight_shift=1.0, dropout=0.1),
               dict(pre="layer", gate="channel"), dict(post="layer", gate="full", gate_sigmoid=True),
               dict(gate="token")):
        d = mel.Residual(T, H, dtype, **kw)
        prm = {n: new(*s) for n, s in d.param_shapes().items()}
        h, y = new(T, H), new(T, H)
        h[0, :32] = 0
        y[0, :32] = 0
        e = lambda: torch.full_like(h, 7.0)  # noqa: E731
        h1, x1, s1 = e(), e(), torch.empty(T, 4, device="cuda")
        h2, x2, s2 = e(), e(), torch.empty(T, 4, device="cuda")
        mel.moe_residual_norm_fwd(d, h, y, prm, h1, x1, s1, rng=rng)
        want, got, alone = (_blank(mel, T, H, "fp8") for _ in range(3))
        mel.moe_mx_quantize(x1, *want, "fp8")
        mel.moe_residual_norm_mx_fwd(d, h, y, prm, h2, *got, s2, x_out=x2, rng=rng)
        mel.moe_residual_norm_mx_fwd(d, h, y, prm, h2, *alone, None, rng=rng)
        for a, b in ((h1, h2), (x1, x2), (s1, s2), *zip(want, got), *zip(want, alone)):
            assert torch.equal(a, b)
    # no block output, and in place
    d = mel.Residual(T, H, dtype)
    prm = {"w_pre": new(H)}
    x1, got, want = torch.empty_like(h), _blank(mel, T, H, "fp8"), _blank(mel, T, H, "fp8")
    mel.moe_residual_norm_fwd(d, h, None, prm, None, x1, None)
    mel.moe_mx_quantize(x1, *want, "fp8")
    mel.moe_residual_norm_mx_fwd(d, h, None, prm, None, *got, None)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_graph_streams_and_neighbours():
    mel = _mel()
    say("[mx graph]")
    T, H = 77, 2880
    d = mel.Residual(T, H)
    h, y, w = (torch.randn(s, device="cuda").bfloat16() for s in ((T, H), (T, H), (H,)))
    n_s = T * mel.mx_scale_cols(H)
    big_c = torch.full((T * H + 512,), 9, device="cuda", dtype=torch.uint8)
    big_s = torch.full((n_s + 512,), 9, device="cuda", dtype=torch.uint8)
    codes, scales = big_c[256:-256].view(T, H), big_s[256:-256].view(T, -1)
    c4, s4 = _blank(mel, T, H, "fp4")
    back, h_out = torch.empty_like(h), torch.empty_like(h)

    def step(stream=None):
        mel.moe_residual_norm_mx_fwd(d, h, y, {"w_pre": w}, h_out, codes, scales, None, stream=stream)
        mel.moe_mx_quantize(h_out, c4, s4, "fp4", stream=stream)
        mel.moe_mx_dequantize(c4, s4, back, "fp4", stream=stream)

    outs = (codes, scales, c4, s4, back)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        y.mul_(1.25)
        step()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
    for b in (big_c, big_s):
        assert (b[:256] == 9).all() and (b[-256:] == 9).all()
    empty = torch.empty(0, 64, device="cuda")
    mel.moe_mx_quantize(empty, *_blank(mel, 0, 64, "fp4"), "fp4")


def test_refusals():
    mel = _mel()
    x = torch.ones(4, 64, device="cuda")
    c, s = _blank(mel, 4, 64, "fp8")
    with pytest.raises(ValueError, match="codes must have shape"):
        mel.moe_mx_quantize(x, c, s, "fp4")
    with pytest.raises(ValueError, match="scales must have shape"):
        mel.moe_mx_quantize(x, c, s[:, :2].contiguous(), "fp8")
    with pytest.raises(RuntimeError, match="multiple of 32"):
        mel.moe_mx_quantize(torch.ones(4, 48, device="cuda"), *_blank(mel, 4, 48, "fp8"), "fp8")
    with pytest.raises(KeyError):
        mel.moe_mx_quantize(x, c, s, "fp6")
    d = mel.Residual(4, 40)
    h = torch.ones(4, 40, device="cuda").bfloat16()
    with pytest.raises(RuntimeError, match="multiple of 32"):
        mel.moe_residual_norm_mx_fwd(d, h, h.clone(), {"w_pre": h[0]}, torch.empty_like(h),
                                     *_blank(mel, 4, 40, "fp8"), None)

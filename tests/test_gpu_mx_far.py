"""Microscaled rows and weights beyond 32-bit offsets: the last rows and the last expert come out as they
do alone. Values are small integers with scale 1, so that every sum is exact in float32 and results are
compared bit for bit (the largest sum is below 2^24 and no group of eight spans more than 2^13)."""
import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _need(gib):
    free, _ = torch.cuda.mem_get_info()
    if free < gib << 30:
        pytest.skip(f"needs {gib} GiB")


def _fp4(*shape, seed=0):
    """Random E2M1 codes of -2, 0 and 2, packed."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(0, 256, shape, device="cuda", dtype=torch.uint8, generator=g) & 0xEE & 0xCC


def _value4(codes):
    """float64 values of packed E2M1 codes [.., n] -> [.., 2n]."""
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=codes.device, dtype=torch.float64)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return torch.where(c >= 8, -1.0, 1.0) * t[c & 7]


def _scales(mel, *shape):
    return torch.full((*shape[:-1], mel.mx_scale_cols(shape[-1])), 127, device="cuda",
                      dtype=torch.uint8)


@pytest.mark.parametrize("T", [2, 300])
def test_far_expert(T):
    mel = _mel()
    _need(12)
    say(f"[mx far expert] T={T}")
    E, K, N = 40, 8192, 32768     # 128 MiB of codes an expert, 5 GiB in all
    w = torch.zeros(E, N, K // 2, device="cuda", dtype=torch.uint8)
    w[-1] = _fp4(N, K // 2, seed=1)
    a = _fp4(T, K // 2, seed=2)
    sh = mel.MXLinear(T, K, N, a_format="fp4", E=E, k=1)
    offsets = torch.zeros(E + 1, device="cuda", dtype=torch.int32)
    offsets[-1] = T
    y = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    mel.moe_mx_linear(sh, a, _scales(mel, T, K), w, _scales(mel, E, N, K), y, offsets=offsets)
    torch.cuda.synchronize()
    va = _value4(a).float()
    for lo in range(0, N, 4096):
        ref = (va @ _value4(w[-1, lo:lo + 4096]).float().t().contiguous()).bfloat16()
        assert torch.equal(y[:, lo:lo + 4096], ref)


@pytest.mark.parametrize("out", ["bf16", "mx8"])
def test_far_rows(out):
    mel = _mel()
    _need(12)
    T, K, N, last = (1 << 20) + 77, 4128, 32, 333     # 2 GiB of codes and more
    say(f"[mx far rows] {out}")
    a = torch.zeros(T, K // 2, device="cuda", dtype=torch.uint8)
    a[-last:] = _fp4(last, K // 2, seed=3)
    w = _fp4(N, K // 2, seed=4)
    sa, sw = _scales(mel, T, K), _scales(mel, N, K)
    mx = out == "mx8"
    y = torch.empty(T, N, device="cuda", dtype=torch.uint8 if mx else torch.bfloat16)
    ys = torch.empty(T, mel.mx_scale_cols(N), device="cuda", dtype=torch.uint8) if mx else None
    mel.moe_mx_linear(mel.MXLinear(T, K, N, a_format="fp4", out=out), a, sa, w, sw, y, y_scales=ys)
    torch.cuda.synchronize()
    ref = _value4(a[-last:]).float() @ _value4(w).float().t().contiguous()
    if mx:
        got = torch.empty(last, N, device="cuda", dtype=torch.float32)
        mel.moe_mx_dequantize(y[-last:].contiguous(), ys[-last:].contiguous(), got, "fp8")
        codes, scales = torch.empty_like(y[-last:]), torch.empty_like(ys[-last:])
        back = torch.empty_like(got)
        mel.moe_mx_quantize(ref.contiguous(), codes, scales, "fp8")
        mel.moe_mx_dequantize(codes, scales, back, "fp8")
        torch.cuda.synchronize()
        assert torch.equal(got, back)
        assert (y[:-last] == 0).all() and (ys[:-last] == 0).all()
    else:
        assert torch.equal(y[-last:], ref.bfloat16())
        assert (y[:-last] == 0).all()


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_far_conversions(fmt):
    mel = _mel()
    _need(32)
    say(f"[mx far conversions] {fmt}")
    rows, cols, last = (1 << 21) + 5, 2080, 64     # more than 2^32 elements
    x = torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x[-last:] = torch.randn(last, cols, device="cuda", generator=g).bfloat16()
    width = cols if fmt == "fp8" else cols // 2
    codes = torch.empty(rows, width, device="cuda", dtype=torch.uint8)
    scales = torch.empty(rows, mel.mx_scale_cols(cols), device="cuda", dtype=torch.uint8)
    mel.moe_mx_quantize(x, codes, scales, fmt)
    few, few_s = torch.empty_like(codes[-last:]), torch.empty_like(scales[-last:])
    mel.moe_mx_quantize(x[-last:].contiguous(), few, few_s, fmt)
    torch.cuda.synchronize()
    assert torch.equal(codes[-last:], few) and torch.equal(scales[-last:], few_s)
    x.fill_(7)
    mel.moe_mx_dequantize(codes, scales, x, fmt)
    back = torch.empty(last, cols, device="cuda", dtype=torch.bfloat16)
    mel.moe_mx_dequantize(few, few_s, back, fmt)
    torch.cuda.synchronize()
    assert torch.equal(x[-last:], back) and (x[:-last] == 0).all()

"""The sums of the products: float32's by default, and with `fast` those of one matrix instruction.

test_small_codes_beside_large_ones: eight neighbours 448 w - 448 w + c w, for every finite E4M3 code c and
every E2M1 code w. All are multiples of 2^-10 of magnitude at most 2688, and the float32 sums of the eight,
in any order that keeps the codes of 4 and more apart from the others, are exact: 448 w - 448 w (+ c w)
needs 2688 / 2^-2 < 2^14 steps, c w alone 6 bits. So the result is c w itself, which every 16-bit type
holds (6 bits from 2^-10 on). With an 8-bit result it is the code that moe_mx_quantize's oracle gives.

test_fast: the forms of test_gpu_mx_linear.py and its derived tolerances, which allow what one instruction
cuts off."""
import functools

import numpy as np
import pytest
import torch

import test_gpu_mx_linear as base
from gpu_util import say
from oracle import microscale as X

pytestmark = pytest.mark.gpu


def _rows(fmt_codes, where, K):
    """[len(codes), K] codes: 448, -448 and the code, in one group of eight from `where` on."""
    a = np.zeros((len(fmt_codes), K), np.uint8)
    a[:, where] = 0x7e
    a[:, where + 3] = 0xfe
    a[:, where + 6] = fmt_codes
    return a


@pytest.mark.parametrize("reps,N", [(1, 32), (5, 1600), (9, 3104), (9, 6272), (9, 7232)])
@pytest.mark.parametrize("out", ["bf16", "f16", "mx8"])
@pytest.mark.parametrize("where", [0, 24, 120, 568])
def test_small_codes_beside_large_ones(reps, N, out, where):
    mel = base._mel()
    say(f"[mx_linear sums] reps={reps} N={N} {out} at {where}")
    K = 608
    codes = np.tile(np.array([c for c in range(256) if c & 127 != 127], np.uint8), reps)
    if N == 32:
        codes = np.concatenate([codes[0x38:0x40], codes[:4], codes[0x47:0x4b]])  # 16 rows
    a, T = _rows(codes, where, K), len(codes)
    w_codes = (np.arange(N) % 16).astype(np.uint8)
    w = np.repeat(w_codes[:, None], K, 1)
    one = lambda n: torch.full((n, mel.mx_scale_cols(K)), 127, device="cuda", dtype=torch.uint8)  # noqa: E731
    mx = out == "mx8"
    y = torch.empty(T, N, device="cuda", dtype=torch.uint8 if mx else base.DT[out])
    ys = torch.empty(T, mel.mx_scale_cols(N), device="cuda", dtype=torch.uint8) if mx else None
    mel.moe_mx_linear(mel.MXLinear(T, K, N, out=out), torch.from_numpy(a).cuda(), one(T),
                      torch.from_numpy(X.pack(w, "fp4")).cuda(), one(N), y, y_scales=ys)
    torch.cuda.synchronize()
    value = lambda c, fmt: X.dequantize(c[:, None].repeat(32, 1), np.full((len(c), 16), 127, np.uint8),  # noqa: E731
                                        fmt)[:, 0]
    ref = value(codes, "fp8")[:, None] * value(w_codes, "fp4")[None]
    if mx:
        want, want_s = X.quantize(ref, "fp8")
        got, got_s = y.cpu().numpy(), ys.cpu().numpy()
        assert np.array_equal(got_s, want_s)
        # zeros may have either sign
        assert (((got ^ want) == 0) | ((got | want) & 127 == 0)).all()
    else:
        assert np.array_equal(y.double().cpu().numpy(), ref)


def _fast(monkeypatch):
    mel = base._mel()
    monkeypatch.setattr(mel, "MXLinear", functools.partial(mel.MXLinear, fast=True))


@pytest.mark.parametrize("tile", [64, 128, 192, 256])
@pytest.mark.parametrize("out", ["bf16", "f16", "mx8"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_fast(monkeypatch, tile, out, act):
    T, N = {64: (900, 1600), 128: (1100, 3136), 192: (2300, 8352), 256: (2056, 6272)}[tile]
    if act == "swiglu":
        if tile == 192:
            return  # not for SwiGLU
        N //= 2
    _fast(monkeypatch)
    base.check(T, 160, N, "fp8", out, act)


@pytest.mark.parametrize("T,K,N", [(1, 2880, 320), (16, 160, 96), (33, 544, 32)])
@pytest.mark.parametrize("out", ["bf16", "f16", "mx8"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_fast_few_rows(monkeypatch, T, K, N, out, act):
    _fast(monkeypatch)
    base.check(T, K, N, "fp8", out, act)


@pytest.mark.parametrize("T,K,N,out,act,E,k", [
    (300, 1184, 320, "f16", "none", 6, 3), (1100, 1056, 768, "mx8", "swiglu", 4, 2),
    (1500, 1056, 2240, "mx8", "swiglu", 3, 2), (2056, 1056, 4128, "mx8", "none", 2, 2)])
def test_fast_experts(monkeypatch, T, K, N, out, act, E, k):
    _fast(monkeypatch)
    base.check(T, K, N, "fp8", out, act, E, k, True)


def test_fast_changes_nothing_in_4_bits():
    mel = base._mel()
    say("[mx_linear fast fp4]")
    rng = np.random.default_rng(1)
    t = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    a, a_s, _ = base._operand(rng, (300, 608), "fp4")
    w, w_s, _ = base._operand(rng, (320, 608), "fp4")
    y = [torch.empty(300, 320, device="cuda", dtype=torch.float16) for _ in range(2)]
    for fast in (False, True):
        mel.moe_mx_linear(mel.MXLinear(300, 608, 320, "fp4", "f16", fast=fast), t(a), t(a_s), t(w), t(w_s),
                          y[fast])
    assert torch.equal(*y)


def test_layers_take_the_choice():
    mel = base._mel()
    shape, router = mel.Shape(4, 64, 32, 8, 2, 4), mel.GroupedRouter(8, 2)
    for fast in (False, True):
        sub = mel.MoEMXSublayer(shape, router, 32, fast=fast)
        for x in (sub.layer.experts, sub.layer.shared):
            assert x.up.fast is fast and x.down.fast is fast

"""Variants that the smaller cases of grouped routing, of the norm with an 8-bit output and of the
microscaled products do not reach: many tokens, whose rows share a wave; rows of 4096; every format and
output with every tile size. Tolerances are those of the tests they extend."""
import numpy as np
import pytest
import torch

import test_gpu_mx
import test_gpu_mx_linear
import test_gpu_route_grouped as R
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,groups,keep", [
    (4100, 256, 8, 8, 3), (4097, 128, 16, 16, 5), (4099, 64, 8, 1, 1), (4098, 32, 6, 4, 2),
    (4111, 5, 5, 5, 5), (4097, 200, 9, 10, 4), (4101, 34, 2, 2, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_routing_of_many_tokens(T, E, k, groups, keep, score):
    mel = R._mel()
    say(f"[route_grouped many] T={T} E={E} k={k} {groups}/{keep} {score}")
    rng = np.random.default_rng(T + E)
    logits = (rng.normal(size=(T, E)) * 2).astype(np.float32)
    bias = (rng.normal(size=E) * 0.05).astype(np.float32)
    R.run(mel.GroupedRouter(E, k, score, groups, keep, 2, True, 2.5), logits, bias)
    R.run(mel.GroupedRouter(E, k, score, groups, keep, 1, False, -0.5), logits, None)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [32, 48, 100, 256])
def test_routing_of_many_special_tokens(score, E):
    """Ties, masks, rows of nothing and NaN: 64 rows alone, and the same rows 66 times over."""
    mel = R._mel()
    say(f"[route_grouped many special] E={E} {score}")
    rng = np.random.default_rng(5)
    T, k = 64, 6
    tied = rng.integers(-2, 3, size=(T, E)).astype(np.float32)
    masked = rng.normal(size=(T, E)).astype(np.float32)
    masked[rng.random(size=(T, E)) < 0.7] = -np.inf
    masked[3], masked[4, 1:] = -np.inf, -np.inf
    low = np.full((T, E), -np.finfo(np.float32).max, np.float32)
    low[:, 5:9] = rng.normal(size=(T, 4))
    nan = tied.copy()
    nan[:, 3], nan[5] = np.nan, np.nan
    bias = torch.from_numpy(np.round(rng.normal(size=E) * 2).astype(np.float32) / 4).cuda()
    dw = torch.from_numpy(rng.normal(size=(T, k)).astype(np.float32)).cuda()

    def both(r, l, d, b):
        ids = torch.empty(len(l), k, device="cuda", dtype=torch.int32)
        w, dl = torch.empty(len(l), k, device="cuda"), torch.empty_like(l)
        mel.moe_route_grouped(r, l, ids, w, bias=b)
        mel.moe_route_grouped_bwd(r, l, ids, d, dl)
        return ids, w, dl

    for logits in (tied, masked, low, nan):
        l = torch.from_numpy(logits).cuda()
        for renorm in (True, False):
            for groups, keep in ((1, 1), (4, 2)):
                for b in (None, bias):
                    r = mel.GroupedRouter(E, k, score, groups, keep, 2, renorm, 1.0)
                    few = both(r, l, dw, b)
                    many = [v.view(66, T, -1) for v in both(r, l.repeat(66, 1), dw.repeat(66, 1), b)]
                    for v in many:  # the same row gives the same answer everywhere
                        assert torch.equal(v.nan_to_num(9.0), v[:1].expand_as(v).nan_to_num(9.0))
                    assert torch.equal(few[0], many[0][0])
                    assert torch.allclose(few[1], many[1][0], rtol=1e-5, atol=1e-9, equal_nan=True)
                    assert torch.allclose(few[2], many[2][0], rtol=1e-4, atol=2e-6, equal_nan=True)


@pytest.mark.parametrize("T", [1, 33])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_norm_of_4096(T, dtype):
    test_gpu_mx.test_norm_in_8_bits(T, 4096, dtype)


@pytest.mark.parametrize("tile", [64, 128, 192, 256])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("out", ["bf16", "f16", "mx8"])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_products_of_every_kind(tile, fmt, out, act):
    T, N = {64: (900, 1600), 128: (1100, 3136), 192: (2300, 8352), 256: (2056, 6272)}[tile]
    if act == "swiglu":
        if tile == 192:
            return  # not for SwiGLU
        N //= 2
    test_gpu_mx_linear.check(T, 160, N, fmt, out, act)

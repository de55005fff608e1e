"""The float64 oracles of grouped routing, clipping and the microscaled formats: against brute force,
closed forms, central differences and torch's own conversion to 8 bits."""
import itertools

import numpy as np
import pytest
import torch

from oracle import grouped as G
from oracle import microscale as X


def test_choice_against_enumeration():
    """Every set of topk_groups groups and k experts: the chosen one has the largest sums."""
    rng = np.random.default_rng(1)
    E, groups, k = 8, 4, 3
    for score, top in itertools.product(("softmax", "sigmoid"), (1, 2)):
        logits, bias = rng.normal(size=(20, E)), rng.normal(size=E) * 0.2
        v = G.scores(logits, score) + bias
        ids = G.choose(logits, k, score, groups, 2, top, bias)
        for t in range(20):
            part = v[t].reshape(groups, 2)
            gs = np.sort(part, 1)[:, ::-1][:, :top].sum(1)
            kept = max(itertools.combinations(range(groups), 2), key=lambda c: gs[list(c)].sum())
            ok = [e for e in range(E) if e // 2 in kept]
            best = max(itertools.combinations(ok, k), key=lambda c: v[t, list(c)].sum())
            assert set(ids[t]) == set(best)
            assert list(v[t, ids[t]]) == sorted(v[t, ids[t]], reverse=True)


def test_ties_go_to_the_lower_index():
    z = np.zeros((1, 8))
    assert list(G.choose(z, 3, "softmax")[0]) == [0, 1, 2]
    assert list(G.choose(z, 3, "sigmoid", groups=4, topk_groups=2)[0]) == [0, 1, 2]


def test_masked_rows():
    l = np.full((2, 6), -np.inf)
    l[1, 4] = 1.0
    for score in ("softmax", "sigmoid"):
        ids = G.choose(l, 2, score)
        assert list(ids[0]) == [0, 1] and list(ids[1]) == [4, 0]
        for renorm in (False, True):
            w = G.weights(l, ids, score, renorm, 2.0)
            assert list(w[0]) == [0.0, 0.0] and w[1, 1] == 0.0 and w[1, 0] > 0
            assert np.isfinite(G.weights_backward(l, ids, np.ones((2, 2)), score, renorm, 2.0)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_by_differences(score, renorm):
    rng = np.random.default_rng(2)
    logits, dw = rng.normal(size=(5, 9)), rng.normal(size=(5, 4))
    ids = G.choose(logits, 4, score)
    got = G.weights_backward(logits, ids, dw, score, renorm, 2.5)
    step = 1e-6
    for t, e in itertools.product(range(5), range(9)):
        hi, lo = logits.copy(), logits.copy()
        hi[t, e] += step
        lo[t, e] -= step
        d = ((G.weights(hi, ids, score, renorm, 2.5) - G.weights(lo, ids, score, renorm, 2.5)) * dw).sum()
        assert abs(d / (2 * step) - got[t, e]) < 1e-8


def test_renormalised_weights_far_below_zero():
    """Ratios of sigmoids that underflow: e^(l_j - l_i) for very negative logits."""
    l = np.array([[-900.0, -901.0, -2000.0]])
    w = G.weights(l, np.array([[0, 1]]), "sigmoid", True, 1.0)
    assert np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.e)]], rtol=1e-12)


def test_clip():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    norm, out = G.clip(g, 1.0, 0.0)
    assert norm == 5.0 and np.allclose(out[0], [0.6, 0.0]) and np.allclose(out[1], 0.8)
    assert np.array_equal(G.clip(g, 10.0)[1][0], g[0])


def test_tables():
    assert list(X.TABLE["fp4"]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(X.TABLE["fp8"], codes.view(torch.float8_e4m3fn).double().numpy())
    for fmt, top in X.TOP.items():
        assert 2.0 ** top <= X.TABLE[fmt][-1] < 2.0 ** (top + 1)


def test_fp8_codes_against_torch():
    """Blocks whose scale is 1 (largest magnitude 256 to 448): torch's conversion to E4M3."""
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(64, 96)) * np.exp2(rng.integers(-12, 6, size=(64, 96)))).astype(np.float32)
    x = np.clip(x, -440, 440)
    x[:, ::32] = 300.0
    codes, scales = X.quantize(x, "fp8")
    assert (scales[:, :3] == 127).all() and (scales[:, 3:] == 0).all()
    assert np.array_equal(codes, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_rounding(fmt):
    """Every code comes back as itself, every midpoint goes to the even code, and no element is
    off by more than half the step above it."""
    t = X.TABLE[fmt]
    full = np.concatenate([t, -t[1:], [t[-1]] * ((1 - 2 * len(t)) % 32)])
    x = full.reshape(-1, 32).copy()
    x[:, 0] = t[-1]
    codes, scales = X.quantize(x, fmt)
    assert np.array_equal(X.dequantize(codes, scales, fmt), x)
    for i, mid in enumerate((t[1:] + t[:-1]) / 2):
        b = np.full((1, 32), mid)
        b[0, 0] = t[-1]
        assert X.quantize(b, fmt)[0][0, 5] == (i if i % 2 == 0 else i + 1)
    rng = np.random.default_rng(4)
    x = rng.normal(size=(50, 64)) * np.exp2(rng.integers(-30, 30, size=(50, 1)))
    y = X.dequantize(*X.quantize(x, fmt), fmt)
    amax = np.abs(x.reshape(50, 2, 32)).max(2).repeat(32, 1).reshape(50, 64)
    # what stops at the largest code loses most: amax reaches just below 2^(top + 1); half the last
    # step (1 of 5, 16 of 272) is less
    worst = 1 - t[-1] / 2.0 ** (X.TOP[fmt] + 1)
    assert (np.abs(y - x) <= worst * amax).all()


def test_special_blocks():
    x = np.zeros((4, 64))
    x[0, 3], x[1, 40], x[2, 0] = np.nan, -np.inf, 2.0 ** -149
    for fmt in ("fp4", "fp8"):
        codes, scales = X.quantize(x, fmt)
        v = X.dequantize(codes, scales, fmt)
        assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 0).all()
        assert np.isnan(v[1, 32:]).all() and (v[1, :32] == 0).all()
        assert scales[2, 0] == 0 and (v[3] == 0).all() and (scales[3] == 0).all()


def test_packing():
    c = np.arange(16, dtype=np.uint8).reshape(1, 16)
    assert list(X.pack(c, "fp4")[0]) == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
    assert np.array_equal(X.unpack(X.pack(c, "fp4"), "fp4"), c)

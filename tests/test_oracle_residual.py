"""The float64 oracle of the residual-stream operators: Philox against the published known
answers, the dropout mask's definition and rate, and every gradient against central differences."""
import numpy as np
import pytest

from oracle import residual as R


@pytest.mark.parametrize("ctr,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(ctr, key, want):
    """The test vectors that the generator's authors publish for ten rounds of 4x32."""
    assert tuple(int(v) for v in R.philox4x32(ctr, key)) == want


def test_mask_is_by_element_and_site():
    a = R.dropout_keep(1000, 0.3, 5, 7, 2)
    assert np.array_equal(a[:13], R.dropout_keep(13, 0.3, 5, 7, 2))   # a prefix is a prefix
    assert np.array_equal(a, R.dropout_keep(1000, 0.3, 5, 9, 0))      # offset + site
    assert not np.array_equal(a, R.dropout_keep(1000, 0.3, 5, 7, 3))
    assert not np.array_equal(a, R.dropout_keep(1000, 0.3, 6, 7, 2))
    assert np.array_equal(R.dropout_keep(64, 0.5, -1, -1, 1), R.dropout_keep(64, 0.5, 2 ** 64 - 1, 0))


@pytest.mark.parametrize("p", [0.05, 0.1, 0.5, 0.9])
def test_mask_rate(p):
    """Dropped share of n independent draws: five standard deviations, and the rounding of p."""
    n = 400_000
    got = 1.0 - R.dropout_keep(n, p, 11, 3).mean()
    assert abs(got - p) < 5 * np.sqrt(p * (1 - p) / n) + 2.0 ** -17


def _diff(f, x, dout, step=1e-5):
    """Gradient of sum(f(x) dout) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        hi = (f() * dout).sum()
        x[i] = keep - step
        lo = (f() * dout).sum()
        x[i] = keep
        g[i] = (hi - lo) / (2 * step)
    return g


NORM_CASES = [("none", "rms", "none", False), ("rms", "none", "channel", True),
              ("layer", "layer", "token", True), ("rms", "layer", "full", False),
              ("layer", "rms", "full", True), ("none", "none", "token", False)]


@pytest.mark.parametrize("post,pre,gate,sig", NORM_CASES)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_residual_norm_gradients(post, pre, gate, sig, p):
    rng = np.random.default_rng(3)
    T, H = 4, 8
    h, y = rng.normal(size=(T, H)), rng.normal(size=(T, H))
    prm = {"w_post": rng.normal(size=H), "b_post": rng.normal(size=H), "w_pre": rng.normal(size=H),
           "b_pre": rng.normal(size=H),
           "gate": rng.normal(size={"channel": (H,), "token": (T,)}.get(gate, (T, H)))}
    if post != "layer":
        del prm["b_post"]
    kw = dict(post=post, pre=pre, gate=gate, gate_sigmoid=sig, alpha=0.7, eps=1e-3,
              weight_shift=1.0, drop=(p, 9, 4, 1))
    dh_out, dx_out = rng.normal(size=(T, H)), rng.normal(size=(T, H))
    dout = np.concatenate([dh_out, dx_out], 1)

    def f():
        out = R.residual_norm(h, y, prm, **kw)[0]
        x = out * 0 if pre == "none" else R.norm(out, pre, 1e-3, 1.0 + prm["w_pre"],
                                                 prm["b_pre"] if pre == "layer" else None)
        return np.concatenate([out, x], 1)

    h_out = R.residual_norm(h, y, prm, **kw)[0]
    got = R.residual_norm_bwd(dh_out, None if pre == "none" else dx_out, h_out, y, prm, **kw)
    want = {"dh": _diff(f, h, dout), "dy": _diff(f, y, dout)}
    for n in got:
        if n not in want:
            want[n] = _diff(f, prm[n[1:]], dout)
    for n, g in got.items():
        # central differences of step 1e-5: truncation ~1e-10, cancellation ~1e-16 / 1e-5
        np.testing.assert_allclose(g, want[n], rtol=1e-6, atol=1e-8, err_msg=n)


@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_linear_gradients(kind, p):
    rng = np.random.default_rng(4)
    T, K, N = 3, 8, 16
    x, w, b = rng.normal(size=(T, K)), rng.normal(size=(N, K)), rng.normal(size=N)
    drop = (p, 21, 6, 0)
    dy = rng.normal(size=(T, N))
    z = R.linear(x, w, b, None, kind, drop)[1]
    _, dx, dw, db = R.linear_bwd(dy, x, w, z, kind, drop)
    f = lambda: R.linear(x, w, b, None, kind, drop)[0]  # noqa: E731
    for got, t in ((dx, x), (dw, w), (db, b)):
        np.testing.assert_allclose(got, _diff(f, t, dy), rtol=1e-6, atol=1e-8)

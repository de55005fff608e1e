"""Grouped routing where experts are masked by a logit of -infinity, against the float64 oracle and by
counting: a masked expert is chosen only where the free ones do not suffice, whatever the bias."""
import numpy as np
import pytest

from gpu_util import say
from oracle import grouped as G
from test_gpu_route_grouped import _mel, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,keep", [(64, 32, 6, 1, 1), (300, 32, 6, 4, 2), (5000, 64, 4, 16, 5),
                                               (4500, 200, 8, 8, 3), (90, 320, 12, 20, 4),
                                               (40, 1024, 32, 64, 6), (4100, 16, 2, 16, 6)])
def test_masked_experts_with_a_bias(T, E, k, groups, keep, score):
    mel = _mel()
    say(f"[route_grouped masks] T={T} E={E} k={k} {groups}/{keep} {score}")
    rng = np.random.default_rng(T + E)
    logits = rng.normal(size=(T, E)).astype(np.float32)
    # rows from nearly free to nearly all masked, and groups masked as a whole
    dead = rng.random((T, E)) < rng.choice([0.1, 0.5, 0.9, 0.99], size=(T, 1))
    whole = rng.random((T, groups)) < 0.2
    dead |= np.repeat(whole, E // groups, 1)
    dead[0], dead[1] = True, False
    logits[dead] = -np.inf
    for lift in (0.9, 4.0):
        bias = np.where(rng.random(E) < 0.5, lift, -lift).astype(np.float32)
        for top, b in ((1, bias), (2, bias), (2, None)):
            for renorm in (True, False):
                r = mel.GroupedRouter(E, k, score, groups, keep, top, renorm, 1.0)
                ids, w, _ = run(r, logits, b)
                bad = np.take_along_axis(dead, ids, 1)
                assert (w[bad] == 0).all()
                if groups == 1:
                    assert (bad.sum(1) == np.maximum(0, k - (~dead).sum(1))).all()
        assert (G.choose(logits[:1], k, score, bias=bias)[0] == np.arange(k)).all()

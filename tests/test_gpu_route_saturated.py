"""Grouped routing where scores saturate: unequal logits whose scores are the same number. Without a
bias and without summed scores the logits decide, otherwise the lower index, as the float64 oracle
states it."""
import numpy as np
import pytest

from gpu_util import say
from test_gpu_route_grouped import _mel, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,k,groups,keep", [(20, 16, 4, 1, 1), (4200, 16, 4, 4, 2), (30, 320, 8, 32, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_saturated_scores(T, E, k, groups, keep, score):
    mel = _mel()
    say(f"[route_grouped saturated] T={T} E={E} {groups}/{keep} {score}")
    rng = np.random.default_rng(E)
    # sigmoids that round to 1 in 64 bits; exponentials below its range, behind one expert at 0
    base = 60.0 if score == "sigmoid" else -5000.0
    logits = (base + rng.permuted(np.tile(np.arange(E), (T, 1)), axis=1)).astype(np.float32)
    if score == "softmax":
        logits[np.arange(T), rng.integers(0, E, T)] = 0.0
    for top in (1, 2):
        for bias in (None, np.zeros(E, np.float32)):
            r = mel.GroupedRouter(E, k, score, groups, keep, top, True, 1.0)
            ids, _, _ = run(r, logits, bias)
            if groups == 1 and bias is None:
                assert (ids == np.argsort(-logits, 1)[:, :k]).all()

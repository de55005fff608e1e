"""The float64 oracle of grouped routing at logits of +infinity: the limit of large ones."""
import itertools

import numpy as np

from oracle import grouped as G


def test_infinite_logits_are_the_limit_of_large_ones():
    rng = np.random.default_rng(3)
    l = rng.normal(size=(40, 12))
    up = rng.random((40, 12)) < 0.2
    up[0] = True
    l[rng.random((40, 12)) < 0.2] = -np.inf
    top, large = l.copy(), l.copy()
    top[up], large[up] = np.inf, 1e5
    bias, dw = rng.normal(size=12) * 0.1, rng.normal(size=(40, 4))
    for score, (groups, keep), b in itertools.product(("softmax", "sigmoid"), ((1, 1), (4, 3)), (None, bias)):
        a = G.choose(top, 4, score, groups, keep, 2, b)
        assert np.array_equal(a, G.choose(large, 4, score, groups, keep, 2, b))
        for renorm in (False, True):
            assert np.allclose(G.weights(top, a, score, renorm, 2.0), G.weights(large, a, score, renorm, 2.0),
                               rtol=1e-14, atol=0)
            assert np.allclose(G.weights_backward(top, a, dw, score, renorm, 2.0),
                               G.weights_backward(large, a, dw, score, renorm, 2.0), rtol=1e-13, atol=1e-300)

"""The float64 oracle of grouped routing where scores saturate: by the logits where nothing is added to
the scores, by score plus bias otherwise."""
import numpy as np
import pytest

from oracle import grouped as G


@pytest.mark.parametrize("score,row", [("sigmoid", [40.0, 45.0, 39.0, 44.0]),
                                       ("softmax", [-900.0, -800.0, 0.0, -850.0])])
def test_saturated_scores(score, row):
    l = np.array([row])
    by_logit = sorted(range(4), key=lambda e: -row[e])
    assert list(G.choose(l, 4, score)[0]) == by_logit
    assert list(G.choose(l, 4, score, 2, 2, 1)[0]) == by_logit
    first = max(range(2), key=lambda g: max(row[2 * g:2 * g + 2]))
    assert set(G.choose(l, 2, score, 2, 1, 1)[0]) == {2 * first, 2 * first + 1}
    # v ties: to the lower index
    tied = [0, 1, 2, 3] if score == "sigmoid" else [2, 0, 1, 3]
    assert list(G.choose(l, 4, score, bias=np.zeros(4))[0]) == tied
    assert list(G.choose(l, 4, score, 2, 2, 2)[0]) == tied

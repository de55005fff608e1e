"""The float64 oracle of grouped routing where experts are masked by a logit of -infinity: they stay
behind the others whatever their bias, in their groups' sums too."""
import numpy as np
import pytest

from oracle import grouped as G

INF = np.inf


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_a_bias_does_not_bring_masked_experts_back(score, group_top):
    rng = np.random.default_rng(1)
    E, k = 16, 4
    for masked_bias, free_bias in ((0.9, 0.0), (0.0, -1.5), (50.0, -50.0)):
        logits = rng.normal(size=(200, E))
        dead = np.zeros((200, E), bool)
        for t in range(200):  # k to E - 1 experts stay free
            dead[t, rng.permutation(E)[:rng.integers(1, E - k + 1)]] = True
        logits[dead] = -INF
        bias = np.where(rng.random(E) < 0.5, masked_bias, free_bias)
        ids = G.choose(logits, k, score, bias=bias, group_top=group_top)
        assert not np.take_along_axis(dead, ids, 1).any()
        assert (G.weights(logits, ids, score, True, 1.0) > 0).all()
        # within the kept groups: masked ones only fill up what is missing
        ids = G.choose(logits, k, score, 4, 2, group_top, bias)
        for t in range(200):
            free = sum((~dead[t, g * 4:g * 4 + 4]).sum() for g in set(ids[t] // 4))
            assert (~dead[t, ids[t]]).sum() == min(k, free) or len(set(ids[t] // 4)) < 2


def test_groups_with_masked_experts():
    # groups of two: {free .1, masked}, {masked, masked}, {masked, free .3}, {free -2, free -2}
    logits = np.array([[0.1, -INF, -INF, -INF, -INF, 0.3, -2.0, -2.0]])
    bias = np.full(8, 3.0)
    bias[6:] = -1.0
    for score in ("softmax", "sigmoid"):
        pick = lambda keep, k, b=bias: list(G.choose(logits, k, score, 4, keep, 2, b)[0])  # noqa: E731
        assert pick(1, 2) == [6, 7]
        assert pick(2, 3) == [5, 6, 7] and pick(2, 4) == [5, 6, 7, 4]
        assert pick(3, 6) == [5, 0, 6, 7, 1, 4]
        assert pick(4, 8) == [5, 0, 6, 7, 1, 2, 3, 4]
        assert pick(2, 3, None) == [5, 6, 7]
        # by their largest alone the single free expert's group is as good as any
        assert list(G.choose(logits, 2, score, 4, 2, 1, np.zeros(8))[0]) == [5, 0]


def test_rows_of_nothing_else():
    logits = np.full((1, 8), -INF)
    bias = np.arange(8.0)
    for top in (1, 2):
        assert list(G.choose(logits, 3, "sigmoid", 4, 2, top, bias)[0]) == [0, 1, 2]
        assert list(G.choose(logits, 3, "softmax", 1, 1, top, bias)[0]) == [0, 1, 2]

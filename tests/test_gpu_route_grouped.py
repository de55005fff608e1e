"""GPU parity of grouped routing against the float64 oracle.

Choices are compared exactly: the kernel forms score + bias in 64 bits and compares them to 2^-41,
far below the gaps of random float32 logits; ties come from equal logits, which score alike. Where
scores come closer than that without being equal, the choice is the best up to 2^-40.

Weights are float32 with e = 2^-24. An exponential of l - m has the argument's rounding, e |l - m|,
times its value, and expf is within 2 e of that; a sum over at most 1024 positive terms adds at most
16 e for a lane's own and 6 e across lanes; a divide, a product and 1 + exp add one e each. In all
(48 + 4 D) e of the weight, D the largest |l - m| of the row's chosen (48 + 4 * 24 e where a weight is below
e^-24 of the largest: then it is below 4e-11 and the absolute term below covers it). A gradient
c p_j (D_j - sum_i D_i p_i) has that error in every p: (96 + 8 D) e of its largest terms.
"""
import itertools

import numpy as np
import pytest
import torch

from oracle import grouped as G

from gpu_util import say

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
TINY = 1e-37  # float32's normal range


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _spread(l, ids):
    c = np.take_along_axis(np.asarray(l, np.float64), ids, 1)
    m = np.asarray(l, np.float64).max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        d = np.abs(np.where(np.isfinite(c), c, m) - m)
    return np.nan_to_num(d, nan=0.0).max(1, keepdims=True) + np.abs(np.nan_to_num(c, neginf=0.0)).max(1, keepdims=True)


def nearly_best(ids, v, router):
    """The choice `ids` is the best up to scores that are within 2^-40 of each other. Scores are
    compared to 2^-41 of their value, as documented, so where a bias swamps the scores (a softmax
    of logits tens apart gives 1e-15 beside 0.75) experts closer than that may come in either order;
    float64 sums themselves differ by 2^-53 between two ways of forming a softmax."""
    T, E = v.shape
    size = E // router.groups
    slack = 2.0 ** -40 * np.maximum(1.0, np.abs(v).max())
    for t in range(T):
        assert len(set(ids[t])) == router.k
        gs = np.sort(v[t].reshape(router.groups, size), 1)[:, ::-1][:, :router.group_top].sum(1)
        limit = np.sort(gs)[::-1][router.topk_groups - 1]
        assert (gs[ids[t] // size] >= limit - 2 * slack).all()
        picked = v[t, ids[t]]
        assert (picked[:-1] >= picked[1:] - slack).all()
        sure = np.repeat(gs > limit + 2 * slack, size) if router.groups > 1 else np.ones(E, bool)
        rest = sure & ~np.isin(np.arange(E), ids[t])
        assert (v[t, rest] <= picked[-1] + slack).all()


def run(router, logits, bias=None, dw=None, strict=True):
    """Runs both directions and compares; returns (ids, w, dlogits). strict: the choice is the
    oracle's, expert by expert."""
    mel = _mel()
    T, k = logits.shape[0], router.k
    l = torch.from_numpy(logits).cuda()
    b = None if bias is None else torch.from_numpy(bias).cuda()
    ids = torch.full((T, k), -7, device="cuda", dtype=torch.int32)
    w = torch.full((T, k), 7.0, device="cuda")
    mel.moe_route_grouped(router, l, ids, w, bias=b)
    got_ids, got_w = ids.cpu().numpy().astype(np.int64), w.cpu().double().numpy()
    ref_ids = G.choose(logits, k, router.score, router.groups, router.topk_groups,
                       router.group_top, bias)
    if strict:
        assert np.array_equal(got_ids, ref_ids)
    else:
        nearly_best(got_ids, G.scores(logits, router.score) + (0.0 if bias is None else bias), router)
    scale = float(np.float32(router.scale))
    ref_w = G.weights(logits, got_ids, router.score, router.renorm, scale)
    D = _spread(logits, got_ids)
    assert np.isfinite(got_w).all()
    assert (np.abs(got_w - ref_w) <= (48 + 4 * D) * E24 * np.abs(ref_w) + TINY * abs(scale)).all()
    g = np.random.default_rng(9).normal(size=(T, k)).astype(np.float32) if dw is None else dw
    dl = torch.full(l.shape, 7.0, device="cuda")
    mel.moe_route_grouped_bwd(router, l, ids, torch.from_numpy(g).cuda(), dl)
    got_d = dl.cpu().double().numpy()
    ref_d = G.weights_backward(logits, got_ids, g, router.score, router.renorm, scale)
    p = G.weights(logits, got_ids, router.score, router.renorm, abs(scale))
    term = np.zeros_like(ref_d)
    inner = (np.abs(g) * p).sum(1, keepdims=True) / abs(scale)
    if not router.renorm and router.score == "softmax":
        term = abs(scale) * G.scores(logits, "softmax") * inner
    extra = np.abs(g) + (inner if router.renorm or router.score == "softmax" else 0.0)
    np.put_along_axis(term, got_ids, p * extra, 1)
    assert np.isfinite(got_d).all()
    err = np.abs(got_d - ref_d)
    bound = (96 + 8 * D) * E24 * term + TINY * abs(scale)
    assert (err <= bound).all(), (err - bound).max()
    return got_ids, got_w, got_d


SHAPES = [  # T, E, k, groups, topk_groups
    (1, 256, 8, 8, 4), (3, 256, 8, 8, 4), (17, 128, 8, 1, 1), (1000, 256, 8, 8, 3), (65, 32, 4, 4, 2),
    (5, 1, 1, 1, 1), (33, 5, 5, 5, 5), (40, 64, 16, 2, 1), (40, 64, 17, 2, 2), (9, 96, 32, 3, 2),
    (7, 257, 3, 1, 1), (12, 1024, 32, 64, 16), (50, 320, 6, 40, 7), (129, 100, 7, 20, 2),
    (31, 34, 2, 17, 3), (257, 33, 9, 3, 1), (20, 192, 1, 12, 1),
]


@pytest.mark.parametrize("T,E,k,groups,keep", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_parity(T, E, k, groups, keep, score):
    mel = _mel()
    say(f"[route_grouped] T={T} E={E} k={k} {groups}/{keep} {score}")
    rng = np.random.default_rng(T * 1000 + E)
    logits = (rng.normal(size=(T, E)) * 2).astype(np.float32)
    bias = (rng.normal(size=E) * 0.05).astype(np.float32)
    for top, renorm, b in itertools.product((1, 2), (True, False), (None, bias)):
        r = mel.GroupedRouter(E, k, score, groups, keep, top, renorm, 2.5 if renorm else -0.5)
        run(r, logits, b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_masks_and_extremes(score):
    """Equal logits, masked experts, rows with fewer than k left, rows of nothing, large values."""
    mel = _mel()
    say(f"[route_grouped special] {score}")
    rng = np.random.default_rng(5)
    T, E, k = 64, 32, 6
    tied = rng.integers(-2, 3, size=(T, E)).astype(np.float32)
    masked = rng.normal(size=(T, E)).astype(np.float32)
    masked[rng.random(size=(T, E)) < 0.7] = -np.inf
    masked[3], masked[4, 1:] = -np.inf, -np.inf
    low = np.full((T, E), -np.finfo(np.float32).max, np.float32)
    low[:, 5:9] = rng.normal(size=(T, 4))
    far = (rng.normal(size=(T, E)) * 30 - 300).astype(np.float32)
    for logits in (tied, masked, low, far):
        for renorm in (True, False):
            for groups, keep in ((1, 1), (4, 2)):
                for bias in (None, np.round(rng.normal(size=E) * 2).astype(np.float32) / 4):
                    r = mel.GroupedRouter(E, k, score, groups, keep, 2, renorm, 1.0)
                    ids, w, _ = run(r, logits, bias, strict=logits is not far)
                    dead = ~np.isfinite(np.take_along_axis(logits, ids, 1))
                    assert (w[dead] == 0).all()
    # the same row everywhere gives the same answer everywhere
    r = mel.GroupedRouter(E, k, score, 4, 2, 2, True, 1.0)
    a = run(r, np.repeat(tied[:1], 1025, 0), dw=np.repeat(rng.normal(size=(1, k)), 1025, 0).astype(np.float32))
    assert all((x == x[:1]).all() for x in a)


def test_nan_logits_stay_in_bounds():
    """A NaN ranks below every other value: the chosen are distinct experts of the row."""
    mel = _mel()
    say("[route_grouped nan]")
    l = torch.randn(20, 16, device="cuda")
    l[:, 3] = float("nan")
    l[5] = float("nan")
    for score in ("softmax", "sigmoid"):
        ids = torch.empty(20, 8, device="cuda", dtype=torch.int32)
        w = torch.empty(20, 8, device="cuda")
        mel.moe_route_grouped(mel.GroupedRouter(16, 8, score, 4, 2), l, ids, w)
        mel.moe_route_grouped_bwd(mel.GroupedRouter(16, 8, score, 4, 2), l, ids, w, torch.empty_like(l))
        got = ids.cpu().numpy()
        assert ((got >= 0) & (got < 16)).all() and all(len(set(r)) == 8 for r in got)
    ids = torch.empty(20, 8, device="cuda", dtype=torch.int32)
    mel.moe_route_grouped(mel.GroupedRouter(16, 8, "sigmoid"), l, ids, w)
    keep = torch.arange(20) != 5
    assert (ids.cpu()[keep] != 3).all() and torch.isfinite(w.cpu()[keep]).all()


def test_matches_the_plain_router():
    """Without groups, bias and scale it is moe_route of the same kind: ids equal, weights to a
    few roundings."""
    mel = _mel()
    say("[route_grouped plain]")
    l = torch.randn(3000, 128, device="cuda")
    for plain, kw in (("softmax_topk", dict(score="softmax", renorm=False)),
                      ("softmax_topk_renorm", dict(score="softmax")),
                      ("topk_softmax", dict(score="softmax")),
                      ("sigmoid_topk_renorm", dict(score="sigmoid"))):
        out = [(torch.empty(3000, 8, device="cuda", dtype=torch.int32),
                torch.empty(3000, 8, device="cuda"), torch.empty_like(l)) for _ in range(2)]
        dw = torch.randn(3000, 8, device="cuda")
        mel.moe_route(l, 8, plain, out[0][0], out[0][1])
        mel.moe_route_bwd(l, out[0][0], dw, 8, plain, out[0][2])
        r = mel.GroupedRouter(128, 8, **kw)
        mel.moe_route_grouped(r, l, out[1][0], out[1][1])
        mel.moe_route_grouped_bwd(r, l, out[1][0], dw, out[1][2])
        assert torch.equal(out[0][0], out[1][0])
        assert torch.allclose(out[0][1], out[1][1], rtol=1e-5, atol=1e-9)
        assert torch.allclose(out[0][2], out[1][2], rtol=1e-4, atol=2e-6)


def test_graph_streams_and_neighbours():
    mel = _mel()
    say("[route_grouped graph]")
    r = mel.GroupedRouter(256, 8, "sigmoid", 8, 4, scale=2.5)
    T = 333
    l, bias, dw = torch.randn(T, 256, device="cuda"), torch.randn(256, device="cuda") * 0.1, \
        torch.randn(T, 8, device="cuda")
    big_i = torch.full((T * 8 + 64,), -9, device="cuda", dtype=torch.int32)
    big_d = torch.full((T * 256 + 64,), 9.0, device="cuda")
    ids, w, dl = big_i[32:-32].view(T, 8), torch.empty(T, 8, device="cuda"), big_d[32:-32].view(T, 256)

    def step(stream=None):
        mel.moe_route_grouped(r, l, ids, w, bias=bias, stream=stream)
        mel.moe_route_grouped_bwd(r, l, ids, dw, dl, stream=stream)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(3):
        l.copy_(torch.randn(T, 256, generator=torch.Generator().manual_seed(seed)))
        step()
        want = [t.clone() for t in (ids, w, dl)]
        for t in (ids, w, dl):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (ids, w, dl)))
    assert (big_i[:32] == -9).all() and (big_i[-32:] == -9).all()
    assert (big_d[:32] == 9).all() and (big_d[-32:] == 9).all()

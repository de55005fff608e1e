"""Grouped routing at logits of +infinity against the float64 oracle: they are chosen first, share a
softmax in equal parts, and no weight or gradient of their row is NaN.

Tolerances are those of test_gpu_route_grouped.py, (48 + 4 D) e of a weight and (96 + 8 D) e of a
gradient's largest terms with e = 2^-24; the finite logits are normal and below 7 in magnitude, so D, the
largest distance and magnitude of the chosen, is at most 21. At an infinite one the exponentials are 0
and 1 without any rounding."""
import numpy as np
import pytest
import torch

from gpu_util import say
from oracle import grouped as G
from test_gpu_route_grouped import E24, TINY, _mel

pytestmark = pytest.mark.gpu

D = 21


@pytest.mark.parametrize("T,E,k,groups,keep", [(60, 16, 4, 1, 1), (4200, 32, 4, 8, 3), (50, 320, 8, 32, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinite_logits(T, E, k, groups, keep, score):
    mel = _mel()
    say(f"[route_grouped infinite] T={T} E={E} {groups}/{keep} {score}")
    rng = np.random.default_rng(T)
    logits = rng.normal(size=(T, E)).astype(np.float32)
    logits[rng.random((T, E)) < 0.1] = -np.inf
    up = rng.random((T, E)) < rng.choice([0.0, 0.02, 0.3], size=(T, 1))
    up[0] = True
    logits[up] = np.inf
    assert np.abs(logits[np.isfinite(logits)]).max() < 7
    bias = (np.arange(E) % 7 / 64).astype(np.float32)
    g = rng.normal(size=(T, k)).astype(np.float32)
    l, gt = torch.from_numpy(logits).cuda(), torch.from_numpy(g).cuda()
    for top in (1, 2):
        for b in (None, bias):
            for renorm in (True, False):
                r = mel.GroupedRouter(E, k, score, groups, keep, top, renorm, 2.0)
                ids = torch.empty(T, k, device="cuda", dtype=torch.int32)
                w, dl = torch.empty(T, k, device="cuda"), torch.empty_like(l)
                mel.moe_route_grouped(r, l, ids, w, bias=None if b is None else torch.from_numpy(b).cuda())
                mel.moe_route_grouped_bwd(r, l, ids, gt, dl)
                got, w, dl = ids.cpu().numpy().astype(np.int64), w.cpu().double().numpy(), dl.cpu().double().numpy()
                assert np.array_equal(got, G.choose(logits, k, score, groups, keep, top, b))
                ref = G.weights(logits, got, score, renorm, 2.0)
                assert (np.abs(w - ref) <= (48 + 4 * D) * E24 * ref + TINY).all()
                if score == "softmax" and groups == 1:
                    want = np.where(up.any(1), np.minimum(up.sum(1), k), k)
                    assert ((w > 0).sum(1) <= want).all()
                inner = (np.abs(g) * ref).sum(1, keepdims=True)
                term = G.scores(logits, score) * inner
                np.put_along_axis(term, got, ref * np.abs(g) + ref * inner, 1)
                exact = G.weights_backward(logits, got, g, score, renorm, 2.0)
                assert (np.abs(dl - exact) <= (96 + 8 * D) * E24 * term + TINY).all()

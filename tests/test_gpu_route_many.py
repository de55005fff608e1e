"""Grouped routing of more tokens than one grid's 2^32 threads take: the first, the last and the rows
around the border of the launches come out as they do alone."""
import pytest
import torch

from gpu_util import say
from test_gpu_route_grouped import _mel

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E,groups,part", [((1 << 28) + 5, 2, 1, 1 << 27), ((1 << 26) + 5, 17, 17, 1 << 25)])
def test_more_tokens_than_a_grid_holds(T, E, groups, part):
    mel = _mel()
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GiB")
    say(f"[route_grouped many] T={T} E={E} groups={groups}")
    r = mel.GroupedRouter(E, 1, "sigmoid", groups, groups, renorm=False)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    logits = torch.randn(T, E, device="cuda", generator=gen)
    bias = torch.zeros(E, device="cuda")
    ids = torch.full((T, 1), -7, device="cuda", dtype=torch.int32)
    w = torch.full((T, 1), 7.0, device="cuda")
    mel.moe_route_grouped(r, logits, ids, w, bias=bias)
    dl = torch.full_like(logits, 7.0)
    mel.moe_route_grouped_bwd(r, logits, ids, w, dl)
    torch.cuda.synchronize()
    spans = [(0, 5000), (T - 5000, T)] + [(b - 2500, min(b + 2500, T)) for b in range(part, T, part)]
    for lo, hi in spans:
        l = logits[lo:hi].clone()
        i1, w1, d1 = torch.empty_like(ids[lo:hi]), torch.empty_like(w[lo:hi]), torch.empty_like(l)
        mel.moe_route_grouped(r, l, i1, w1, bias=bias)
        mel.moe_route_grouped_bwd(r, l, i1, w1, d1)
        torch.cuda.synchronize()
        assert torch.equal(ids[lo:hi], i1) and torch.equal(w[lo:hi], w1) and torch.equal(dl[lo:hi], d1)
        assert torch.equal(i1[:, 0].long(), l.argmax(1))
    for lo in range(0, T, 1 << 24):
        assert ((ids[lo:lo + (1 << 24)] >= 0) & (w[lo:lo + (1 << 24)] < 1)).all()

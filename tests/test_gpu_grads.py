"""GPU parity of the gradient norm and clipping against float64.

The norm is summed in 64 bits and rounded to float32 once: within 2^-24 of the value, plus 2^-50 for
the order of the sums. A clipped gradient is its float32 product with the factor, which carries the
norm's rounding and its own (2 e), rounded once more to the product (e) and to the type (u)."""
import numpy as np
import pytest
import torch

from oracle import grouped as G

from gpu_util import say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E24 = 2.0 ** -24


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _ws(mel, lst):
    return torch.empty(max(1, mel.moe_grad_norm_workspace_bytes(lst)), device="cuda", dtype=torch.uint8)


def _norm_and_clip(mel, lst, max_norm, stream=None):
    norm = torch.full((1,), -1.0, device="cuda")
    mel.moe_grad_norm(lst, norm, _ws(mel, lst), stream=stream)
    mel.moe_grad_clip(lst, norm, max_norm, stream=stream)
    return norm


def _check(name, grads, max_norm, out=None):
    mel = _mel()
    src = [g.double().cpu().numpy() for g in grads]
    lst = mel.GradList(grads, out)
    norm = _norm_and_clip(mel, lst, max_norm)
    ref, want = G.clip(src, float(np.float32(max_norm)), float(np.float32(1e-6)))
    assert abs(norm.item() - ref) <= (E24 + 2.0 ** -50) * ref, (name, norm.item(), ref)
    for g, s, w in zip(lst.out, src, want):
        u = torch.finfo(g.dtype).eps / 2
        got = g.double().cpu().numpy()
        tiny = float(torch.finfo(g.dtype).smallest_normal) * torch.finfo(g.dtype).eps
        assert (np.abs(got - w) <= (u + 4 * E24) * np.abs(w) + tiny).all(), name
    if ref < max_norm:
        assert all(np.array_equal(g.double().cpu().numpy(), s) for g, s in zip(lst.out, src))


SIZES = [[1], [7], [0, 3, 0], [16384], [16385], [16384 * 3 + 5, 1, 9], [8, 16, 24] * 30, [1] * 200,
         [2048 * 16384 + 77], [300000] * 81, []]


@pytest.mark.parametrize("i", range(len(SIZES)))
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32", "mixed"])
def test_parity(i, dtype):
    say(f"[grads] {i} {dtype}")
    g = torch.Generator(device="cuda")
    g.manual_seed(i)
    kinds = list(DT.values())
    grads = [torch.randn(n, device="cuda", generator=g).to(kinds[j % 3] if dtype == "mixed" else DT[dtype])
             for j, n in enumerate(SIZES[i])]
    total = sum(SIZES[i]) ** 0.5
    _check("in place", [t.clone() for t in grads], 0.3 * total)
    _check("out", grads, 0.3 * total, [torch.zeros_like(t) for t in grads])
    _check("not clipped", [t.clone() for t in grads], 3 * total + 1)
    if dtype != "f32":
        return
    # off 16-byte boundaries, source and output differently
    odd = [torch.randn(n + 3, device="cuda", generator=g)[3:] for n in SIZES[i][:5]]
    _check("odd", odd, 0.3 * total, [torch.zeros(t.numel() + 1, device="cuda")[1:] for t in odd])


def test_range_of_values():
    """Squares beyond float32's range, tiny gradients beside none, zeros, infinities and NaN."""
    mel = _mel()
    say("[grads range]")
    _check("large", [torch.full((1000,), 3e25, device="cuda"), torch.full((7,), -1e30, device="cuda")], 1.0)
    _check("tiny", [torch.full((1000,), 1e-30, device="cuda")], 1e-35)
    _check("zeros", [torch.zeros(50, device="cuda")], 1.0)
    _check("to zero", [torch.ones(50, device="cuda")], 0.0)
    for bad, kept in ((float("inf"), 0.0), (float("nan"), float("nan"))):
        g = [torch.ones(20, device="cuda"), torch.ones(20, device="cuda")]
        g[1][4] = bad
        norm = _norm_and_clip(mel, mel.GradList(g), 1.0)
        assert norm.isnan() if bad != bad else norm.isinf()
        assert g[1][4].isnan()
        assert g[0].isnan().all() if kept != kept else (g[0] == 0).all()


def test_graph_repeats_and_neighbours():
    mel = _mel()
    say("[grads graph]")
    big = torch.zeros(3, 70000, device="cuda")
    grads = [big[0, 64:50064], big[1, 64:65064], big[2, 64:69]]
    src = [torch.randn_like(t) for t in grads]
    lst = mel.GradList(grads)
    norm, ws = torch.empty(1, device="cuda"), _ws(mel, lst)

    def step(stream=None):
        for t, s in zip(grads, src):
            t.copy_(s)
        mel.moe_grad_norm(lst, norm, ws)
        mel.moe_grad_clip(lst, norm, 1.0)

    step()
    want = [t.clone() for t in (*grads, norm)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (*grads, norm)))
        src[0].mul_(1.5)
        step()
        want = [t.clone() for t in (*grads, norm)]
    assert (big[:, :64] == 0).all() and (big[0, 50064:] == 0).all() and (big[2, 69:] == 0).all()
    # two lists on two streams, with workspaces of their own
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [[torch.randn(100000, device="cuda") for _ in range(3)] for _ in range(2)]
    refs = [G.clip([t.double().cpu().numpy() for t in s], 1.0)[0] for s in sets]
    lists = [mel.GradList(s) for s in sets]
    norms, wss = [torch.empty(1, device="cuda") for _ in range(2)], [_ws(mel, x) for x in lists]
    torch.cuda.synchronize()
    for _ in range(10):
        for j in range(2):
            mel.moe_grad_norm(lists[j], norms[j], wss[j], stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        assert abs(norms[j].item() - refs[j]) <= 2 * E24 * refs[j]


def test_refusals():
    mel = _mel()
    a, b = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="outputs"):
        mel.GradList([a, b], [a])
    with pytest.raises(ValueError, match="contiguous"):
        mel.GradList([torch.ones(8, 8, device="cuda").t()])
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        mel.GradList([torch.ones(8, device="cuda", dtype=torch.int32)])
    norm = torch.ones(1, device="cuda")
    for lst in (mel.GradList([a, a]), mel.GradList([a], [b[:64]]), mel.GradList([a, b], [b, a])):
        if lst.grads == [a] and lst.out[0] is not a:
            mel.moe_grad_clip(lst, norm, 1.0)
            continue
        with pytest.raises(RuntimeError, match="overlaps"):
            mel.moe_grad_clip(lst, norm, 1.0)
    lst = mel.GradList([a])
    with pytest.raises(RuntimeError, match="overlaps"):
        mel.moe_grad_clip(lst, a[:1], 1.0)
    for kw in (dict(max_norm=-1.0), dict(max_norm=float("inf")), dict(max_norm=1.0, eps=0.0)):
        with pytest.raises(RuntimeError):
            mel.moe_grad_clip(lst, norm, **kw)
    a.set_(torch.ones(64, device="cuda"))
    with pytest.raises(ValueError, match="moved"):
        mel.moe_grad_norm(lst, norm, torch.empty(64, device="cuda"))

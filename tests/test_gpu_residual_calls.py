"""Ways of calling the residual-stream operators that a program may take: parameters that are
nn.Parameter, another stream, two calls at once on two streams, the smallest and odd sizes, the same
call twice, and a frozen graph next to eager calls."""
import pytest
import torch

from gpu_util import say
from test_gpu_residual import DT, _rng

pytestmark = pytest.mark.gpu


def _mel():
    import mixture_experts_lora_amd as mel
    return mel


def _new(*s, dtype="bf16", seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(s) + seed)
    return torch.randn(s, device="cuda", generator=g).to(DT[dtype])


def _step(mel, T, H, seed=0, p=0.1):
    """One forward and backward of norm and linear on buffers of its own; returns its outputs."""
    d = mel.Residual(T, H, post="layer", pre="rms", gate="token", gate_sigmoid=True, dropout=p)
    lin = mel.LinearShape(T, H, H, act="gelu", dropout=p)
    h, y = _new(T, H, seed=seed), _new(T, H, seed=seed + 1)
    prm = {n: torch.nn.Parameter(_new(*s, seed=seed + 2), requires_grad=False)
           for n, s in d.param_shapes().items()}
    w, b = torch.nn.Parameter(_new(H, H, seed=seed + 3)), _new(H, seed=seed + 4)
    e = lambda t: torch.empty_like(t, requires_grad=False)  # noqa: E731
    z, pre, h_out, x_out, st = e(h), e(h), e(h), e(h), torch.empty(T, 4, device="cuda")
    dh, dy, dx, dw, db = e(h), e(h), e(h), e(w), e(b)
    grads = {"d" + n: e(t) for n, t in prm.items()}
    wf, wb = (torch.empty(max(1, n), device="cuda", dtype=torch.uint8)
              for n in mel.moe_linear_workspace_bytes(lin))
    wr = torch.empty(mel.moe_residual_norm_workspace_bytes(d), device="cuda", dtype=torch.uint8)
    rng = _rng(seed, 3)

    def run(stream=None):
        kw = dict(rng=rng, stream=stream)
        mel.moe_linear_fwd(lin, y, w.detach(), z, wf, bias=b, residual=h, pre=pre, **kw)
        mel.moe_residual_norm_fwd(d, z, y, prm, h_out, x_out, st, **kw)
        mel.moe_residual_norm_bwd(d, h, x_out, h_out, y, prm, st, dh, dy, grads, wr, **kw)
        mel.moe_linear_bwd(lin, dh, y, w.detach(), pre, dx, dw, db, wb, **kw)

    return run, [z, pre, h_out, x_out, st, dh, dy, dx, dw, db, *grads.values()]


def test_other_streams_and_two_at_once():
    mel = _mel()
    say("[calls streams]")
    sizes = [(300, 584), (777, 264)]
    want, steps = [], []
    for i, (T, H) in enumerate(sizes):
        run, outs = _step(mel, T, H, seed=10 * i)
        run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outs])
        for t in outs:
            t.zero_()
        steps.append((run, outs))
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    for _ in range(20):  # interleaved on two streams, one by argument and one as the current one
        steps[0][0](stream=streams[0])
        with torch.cuda.stream(streams[1]):
            steps[1][0]()
    torch.cuda.synchronize()
    for (run, outs), ref in zip(steps, want):
        for a, b in zip(outs, ref):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,H", [(1, 8), (2, 8), (17, 16), (5, 8192)])
def test_smallest_sizes_twice(T, H):
    mel = _mel()
    say(f"[calls small] T={T} H={H}")
    run, outs = _step(mel, T, H, seed=3)
    run()
    first = [t.clone() for t in outs]
    assert all(torch.isfinite(t).all() for t in first)
    run()
    for a, b in zip(first, outs):
        assert torch.equal(a, b)


def test_neighbours_are_left_alone():
    """Outputs inside larger buffers: what lies before and after them keeps its values."""
    mel = _mel()
    say("[calls neighbours]")
    T, H = 37, 264
    n = T * H
    d = mel.Residual(T, H, pre="layer", dropout=0.2)
    prm = {n_: _new(*s) for n_, s in d.param_shapes().items()}
    big = torch.full((4, n + 1024), 7.0, device="cuda", dtype=torch.bfloat16)
    cut = [b[512:512 + n].view(T, H) for b in big]
    h, y = _new(T, H), _new(T, H, seed=1)
    mel.moe_residual_norm_fwd(d, h, y, prm, cut[0], cut[1], None, rng=_rng())
    lin = mel.LinearShape(T, H, H)
    ws = torch.empty(max(1, mel.moe_linear_workspace_bytes(lin)[0]), device="cuda",
                     dtype=torch.uint8)
    mel.moe_linear_fwd(lin, h, _new(H, H), cut[2], ws, pre=cut[3])
    torch.cuda.synchronize()
    assert (big[:, :512] == 7).all() and (big[:, 512 + n:] == 7).all()
    assert all((c != 7).any() for c in cut)

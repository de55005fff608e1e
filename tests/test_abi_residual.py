"""Refusals of the residual-stream calls on the CPU: every call here fails its argument checks, so
no kernel is ever launched."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_lora_amd import _lib
    return _lib.load()


def at(i):
    return P(0x10000000 + i * 0x1000000)


def desc(T=64, H=128, dtype=1, post=0, pre=1, gate=0, sig=0, alpha=1.0, eps=1e-5, shift=0.0, p=0.0):
    from mixture_experts_lora_amd._lib import MoeResidual
    return MoeResidual(T, H, dtype, post, pre, gate, sig, alpha, eps, shift, p)


def params(**kw):
    from mixture_experts_lora_amd._lib import MoeResidualParams
    v = dict(w_post=0x50000000, b_post=0x51000000, gate=0x52000000, w_pre=0x53000000,
             b_pre=0x54000000)
    v.update(kw)
    return MoeResidualParams(**v)


def err(lib):
    return lib.moe_last_error().decode()


def test_dropout_refusals(lib):
    rng = at(9)
    ok = (1, 64, 0.1, rng, 0, at(0), at(1), None)

    def call(**kw):
        names = ("dtype", "n", "p", "rng", "site", "src", "dst", "stream")
        a = dict(zip(names, ok))
        a.update(kw)
        return lib.moe_dropout(*(a[n] for n in names))

    assert call(dtype=5) == 1
    assert call(n=-1) == 1
    assert call(n=(1 << 40) + 1) == 1
    for p in (-0.1, 1.0, 1.5, float("nan"), 0.99999999):
        assert call(p=p) == 1, p
    assert call(p=1 - 2.0 ** -18) == 1          # rounds to 1 in steps of 2^-16
    assert call(rng=None) == 1
    assert call(rng=P(rng.value + 4)) == 1
    assert "8-byte" in err(lib)
    assert call(src=None) == 1 and call(dst=None) == 1
    assert call(dst=P(at(0).value + 16)) == 1   # partial overlap
    assert "overlaps" in err(lib)
    assert call(dst=P(rng.value - 64), n=64) == 1   # runs over rng
    assert call(n=0, src=None, dst=None) == 0   # nothing to do
    assert call(n=0, p=2.0) == 1                # p is checked all the same


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(H=0), 1), (dict(H=-8), 1), (dict(dtype=3), 1), (dict(post=3), 1),
    (dict(pre=-1), 1), (dict(gate=4), 1), (dict(gate=-1), 1), (dict(eps=-1e-6), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(H=100), 2),
    (dict(H=16392), 2),
])
def test_residual_descriptor(lib, kw, status):
    n = ctypes.c_size_t()
    assert lib.moe_residual_norm_workspace_bytes(ctypes.byref(desc(**kw)), ctypes.byref(n)) == status
    assert err(lib)


def test_residual_workspace(lib):
    n = ctypes.c_size_t()

    def need(**kw):
        assert lib.moe_residual_norm_workspace_bytes(ctypes.byref(desc(**kw)), ctypes.byref(n)) == 0
        return n.value

    assert need(pre=0) == 0
    assert need(T=1) == 128 * 4
    assert need(T=1, pre=2, post=2, gate=1) == 5 * 128 * 4
    # bounded however many tokens: a fixed number of partial rows
    assert need(T=2 ** 31 - 1, H=2880) == need(T=2 ** 20, H=2880) < 1 << 25
    assert lib.moe_residual_norm_workspace_bytes(None, ctypes.byref(n)) == 1
    assert lib.moe_residual_norm_workspace_bytes(ctypes.byref(desc()), None) == 1


def test_residual_forward_refusals(lib):
    def call(d, h=at(0), y=at(1), q=None, rng=None, h_out=at(2), x_out=at(3), stats=at(4)):
        q = params() if q is None else q
        return lib.moe_residual_norm_fwd(ctypes.byref(d), h, y, ctypes.byref(q), rng, 0, h_out,
                                         x_out, stats, None)

    assert call(desc(), h=None, y=None) == 1
    for kw in (dict(post=1), dict(gate=1), dict(p=0.1)):
        assert call(desc(**kw), y=None, rng=at(9)) == 1, kw
        assert "needs y" in err(lib)
    assert call(desc(p=0.1)) == 1                                  # rng
    assert call(desc(p=1.0), rng=at(9)) == 1
    assert call(desc(), q=params(w_pre=None)) == 1
    assert call(desc(post=1), q=params(w_post=None)) == 1
    assert call(desc(gate=2), q=params(gate=None)) == 1
    assert call(desc(), h_out=None) == 1                           # y is there to be added
    assert call(desc(), x_out=None) == 1
    assert call(desc(pre=0)) == 1                                  # x_out without a pre norm
    assert call(desc(pre=0), y=None, h_out=None, x_out=None) == 1  # no output
    for kw in (dict(h=P(0x10000008)), dict(y=P(0x11000002)), dict(h_out=P(0x12000004)),
               dict(x_out=P(0x13000008)), dict(stats=P(0x14000004)),
               dict(q=params(w_pre=0x53000002))):
        assert call(desc(), **kw) == 1, kw
        assert "16-byte" in err(lib)
    assert call(desc(gate=3), q=params(gate=0x52000002)) == 1
    rows = 64 * 128 * 2
    for kw in (dict(x_out=at(2)), dict(x_out=at(0)), dict(x_out=at(1)), dict(h_out=at(1)),
               dict(h_out=P(at(0).value + 16)), dict(stats=P(at(2).value + rows - 16)),
               dict(x_out=P(0x53000000)), dict(h_out=P(0x53000010 - rows))):
        assert call(desc(), **kw) == 1, kw
        assert "overlaps" in err(lib)


def test_residual_backward_refusals(lib):
    from mixture_experts_lora_amd._lib import MoeResidualGrads

    def call(d, dh_out=at(0), dx_out=at(1), h_out=at(2), y=at(3), q=None, stats=at(4), rng=None,
             dh=at(5), dy=at(6), g=(), ws=at(8), ws_bytes=1 << 20):
        q = params() if q is None else q
        g = MoeResidualGrads(**dict(g))
        return lib.moe_residual_norm_bwd(ctypes.byref(d), dh_out, dx_out, h_out, y, ctypes.byref(q),
                                         stats, rng, 0, dh, dy, ctypes.byref(g), ws, ws_bytes, None)

    assert call(desc(), dx_out=None) == 1
    assert call(desc(), h_out=None) == 1
    assert call(desc(), stats=None) == 1
    assert call(desc(pre=0)) == 1                                     # dx_out without a pre norm
    assert call(desc(pre=0), dx_out=None, dh_out=None) == 1
    assert call(desc(post=1), y=None) == 1
    assert call(desc(gate=3), y=None) == 1
    assert call(desc(p=0.5)) == 1
    assert call(desc(), dh=None, dy=None) == 1
    # a gradient of a vector that this operator does not have is no output
    assert call(desc(), dh=None, dy=None, g=dict(dw_post=0x60000000, dgate=0x61000000)) == 1
    assert "no output" in err(lib)
    g = dict(dw_pre=0x60000000)
    assert call(desc(), g=g, ws=None) == 1
    need = ctypes.c_size_t()
    assert lib.moe_residual_norm_workspace_bytes(ctypes.byref(desc()), ctypes.byref(need)) == 0
    assert need.value >= 128 * 4
    assert call(desc(), g=g, ws_bytes=need.value - 1) == 3
    assert "residual workspace needs" in err(lib)
    for kw in (dict(dx_out=P(0x11000004)), dict(dy=P(0x16000002)), dict(ws=P(0x18000004)),
               dict(g=dict(dw_pre=0x60000004))):
        assert call(desc(), **kw) == 1, kw
        assert "16-byte" in err(lib)
    for kw in (dict(dy=at(0)), dict(dy=at(5)), dict(dh=at(1)), dict(dh=P(at(0).value + 16)),
               dict(dy=at(2)), dict(g=dict(dw_pre=0x53000000)), dict(g=dict(dw_pre=at(6).value)),
               dict(g=g, ws=at(6)), dict(dy=at(4))):
        assert call(desc(), **kw) == 1, kw
        assert "overlaps" in err(lib)


def test_python_refusals():
    import torch
    import mixture_experts_lora_amd as mel
    d = mel.Residual(4, 8, "f32")
    t = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="on the GPU"):
        mel.moe_residual_norm_fwd(d, t, t, {"w_pre": torch.zeros(8)}, t, t, None)
    with pytest.raises(ValueError, match="w_pre is required"):
        mel.moe_residual_norm_fwd(d, t, t, {}, t, t, None)
    with pytest.raises(ValueError, match="no such gradient"):
        mel.moe_residual_norm_bwd(mel.Residual(4, 8, "f32", pre="none"), t, None, t, t, {}, None, t,
                                  t, {"dw_pre": t}, None)
    with pytest.raises(ValueError, match="on the GPU"):
        mel.moe_dropout(t, t, 0.1, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="must be float32"):
        mel.moe_dropout(t.double(), t.double(), 0.1, None)
    assert mel.Residual(4, 8, post="layer", gate="token").param_shapes() == {
        "w_post": (8,), "b_post": (8,), "w_pre": (8,), "gate": (4,)}
    with pytest.raises(KeyError):
        mel.Residual(4, 8, pre="batch").c()


def lin(T=64, K=128, N=256, dtype=1, act=0, p=0.0):
    from mixture_experts_lora_amd._lib import MoeLinearShape
    return MoeLinearShape(T, K, N, dtype, act, p)


@pytest.mark.parametrize("T,status", [(1 << 30, 2), ((1 << 31) - 1, 2), ((1 << 30) - 1, 0)])
def test_linear_tokens_fit_a_grid(lib, T, status):
    """16-byte rows keep the tensors below 32 GiB; from 2^30 on a launch may need 2^32 threads."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.moe_linear_workspace_bytes(ctypes.byref(lin(T=T, K=8, N=8)), ctypes.byref(f),
                                          ctypes.byref(b)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(K=0), 1), (dict(N=-8), 1), (dict(dtype=4), 1), (dict(act=5), 1),
    (dict(act=-1), 1), (dict(K=100), 2), (dict(N=12), 2),
    (dict(T=1 << 24, K=1032), 1),                        # x above 32 GiB
    (dict(K=32768, N=32768), 1),                         # w of 2 GiB
    (dict(K=16384, N=32768, dtype=0), 1),
    (dict(K=(1 << 20) + 8, N=8), 2), (dict(N=1 << 21, K=8), 2),
])
def test_linear_shape(lib, kw, status):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.moe_linear_workspace_bytes(ctypes.byref(lin(**kw)), ctypes.byref(f),
                                          ctypes.byref(b)) == status
    assert err(lib)


def test_linear_refusals(lib):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    sh = lin(act=2, p=0.1)
    assert lib.moe_linear_workspace_bytes(ctypes.byref(sh), ctypes.byref(f), ctypes.byref(b)) == 0
    assert lib.moe_linear_workspace_bytes(None, ctypes.byref(f), ctypes.byref(b)) == 1
    f, b = f.value, b.value
    assert b >= 64 * 256 * 2                              # dz

    def fwd(sh=sh, x=at(0), w=at(1), bias=at(2), res=at(3), rng=at(4), y=at(5), pre=at(6),
            ws=at(7), n=f):
        return lib.moe_linear_fwd(ctypes.byref(sh), x, w, bias, res, rng, 0, y, pre, ws, n, None)

    def bwd(sh=sh, dy=at(0), x=at(1), w=at(2), pre=at(3), rng=at(4), dx=at(5), dw=at(6), db=at(7),
            ws=at(8), n=b):
        return lib.moe_linear_bwd(ctypes.byref(sh), dy, x, w, pre, rng, 0, dx, dw, db, ws, n, None)

    for n in ("x", "w", "y", "rng"):
        assert fwd(**{n: None}) == 1, n
    for n in ("dy", "x", "w", "pre", "rng"):
        assert bwd(**{n: None}) == 1, n
    assert bwd(dx=None, dw=None, db=None) == 1
    assert bwd(n=b - 1) == 3 and bwd(ws=None) == 1
    if f:
        assert fwd(n=f - 1) == 3 and fwd(ws=None) == 1
    assert fwd(sh=lin(p=1.0)) == 1 and bwd(sh=lin(p=-0.5)) == 1
    for n in ("x", "w", "bias", "res", "y", "pre"):
        assert fwd(**{n: P(0x70000008)}) == 1 and "16-byte" in err(lib), n
    for n in ("dy", "x", "w", "pre", "dx", "dw", "db", "ws"):
        assert bwd(**{n: P(0x70000008)}) == 1 and "16-byte" in err(lib), n
    for kw in (dict(y=at(0)), dict(y=at(1)), dict(y=at(2)), dict(pre=at(3)), dict(pre=at(5)),
               dict(y=P(at(3).value + 16))):
        assert fwd(**kw) == 1 and "overlaps" in err(lib), kw
    for kw in (dict(dx=at(0)), dict(dx=at(6)), dict(dw=at(1)), dict(db=at(3)), dict(ws=at(5)),
               dict(dx=P(at(2).value + 16))):
        assert bwd(**kw) == 1 and "overlaps" in err(lib), kw


def test_only_the_named_input_may_be_the_output(lib):
    """In place means one input and one output: another input at the same address is read by
    blocks that do not wait for the one that writes it."""
    from mixture_experts_lora_amd._lib import MoeResidualGrads
    B = ctypes.byref

    def overlaps(status, what):
        assert status == 1 and what in err(lib), (status, err(lib))

    # a square product: y over the residual, which x, w or the bias is too
    for T in (1, 2, 16, 300):
        sh = lin(T=T, K=520, N=520)
        f = ctypes.c_size_t()
        assert lib.moe_linear_workspace_bytes(B(sh), B(f), None) == 0

        def fwd(x=at(0), w=at(1), bias=at(2), y=at(3), sh=sh, n=f.value):
            return lib.moe_linear_fwd(B(sh), x, w, bias, at(3), None, 0, y, None, at(7), n, None)

        overlaps(fwd(x=at(3)), "y overlaps x")
        overlaps(fwd(w=at(3)), "y overlaps w")
        overlaps(fwd(bias=at(3)), "y overlaps bias")
    # the stream written over, whose buffer is another input's too
    for kw, q, y, what in ((dict(), {}, at(0), "y"), (dict(), dict(w_pre=at(0).value), at(1), "w_pre"),
                           (dict(gate=2), dict(gate=at(0).value), at(1), "gate"),
                           (dict(post=2), dict(b_post=at(0).value), at(1), "b_post")):
        overlaps(lib.moe_residual_norm_fwd(B(desc(**kw)), at(0), y, B(params(**q)), None, 0, at(0),
                                           at(3), at(4), None), "h_out overlaps " + what)
    for kw, dx, h_out, y, stats, q, what in (
            (dict(), at(0), at(2), at(3), at(4), {}, "dx_out"),
            (dict(), at(1), at(0), at(3), at(4), {}, "h_out"),
            (dict(post=1), at(1), at(2), at(0), at(4), {}, "y"),
            (dict(), at(1), at(2), at(3), at(0), {}, "stats"),
            (dict(gate=3), at(1), at(2), at(3), at(4), dict(gate=at(0).value), "gate")):
        overlaps(lib.moe_residual_norm_bwd(B(desc(**kw)), at(0), dx, h_out, y, B(params(**q)), stats,
                                           None, 0, at(0), at(6), B(MoeResidualGrads()), at(8),
                                           1 << 20, None), "dh overlaps " + what)
    overlaps(lib.moe_dropout(1, 64, 0.1, at(0), 0, at(0), at(0), None), "dst overlaps rng")


@pytest.mark.parametrize("dtype,T,K,N", [(0, 262144, 16384, 16384), (1, 1 << 20, 8192, 8192)])
def test_linear_backward_forms_no_needless_partials(lib, dtype, T, K, N):
    """Enough tiles for every CU: the weight gradient takes its rows in a few slices at most, however
    many bytes they have, and the workspace is a fraction of the activations (16 GiB)."""
    b = ctypes.c_size_t()
    assert lib.moe_linear_workspace_bytes(ctypes.byref(lin(T=T, K=K, N=N, dtype=dtype)), None,
                                          ctypes.byref(b)) == 0
    assert b.value <= 2 * N * K * 4


def test_sizes_past_32_bits_are_refused():
    """ctypes would wrap 2^32 + 8 rows to 8, and the call would leave all others as they were."""
    import mixture_experts_lora_amd as mel
    for d in (mel.Residual((1 << 32) + 8, 8), mel.Residual(8, (1 << 32) + 8),
              mel.LinearShape((1 << 32) + 8, 8, 8), mel.LinearShape(8, (1 << 32) + 8, 8),
              mel.LinearShape(8, 8, (1 << 32) + 8), mel.Residual(1 << 31, 8), mel.Residual(0, 8)):
        with pytest.raises(ValueError, match="must be in"):
            d.c()
        with pytest.raises(ValueError, match="must be in"):
            (mel.moe_linear_workspace_bytes if isinstance(d, mel.LinearShape)
             else mel.moe_residual_norm_workspace_bytes)(d)


def test_calls_run_on_their_tensors_device(monkeypatch):
    """Several GPUs, shown with the binding's calls replaced: a launch happens under the device of
    its tensors, on that device's current stream or the one it is given, and tensors of two devices
    are refused."""
    import contextlib
    import types

    import torch
    import mixture_experts_lora_amd as mel

    class On(torch.Tensor):
        def get_device(self):
            return self.index_

    def on(i):
        t = torch.zeros(1).as_subclass(On)
        t.index_ = i
        return t

    now, log = [0], []

    @contextlib.contextmanager
    def device(i):
        before, now[0] = now[0], i
        yield
        now[0] = before

    monkeypatch.setattr(mel, "_one_gpu", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: types.SimpleNamespace(cuda_stream=100 + now[0]))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)

    def fn(arg, stream):
        log.append((arg, now[0], getattr(stream, "value", stream)))
        return 0

    assert mel._device(None, on(1), None, on(1)) == 1 and mel._device(None) == -1
    with pytest.raises(ValueError, match="tensors on"):
        mel._device(on(0), None, on(1))
    mel._call(fn, "call", 0, None, "a")
    mel._call(fn, "call", 1, None, "b")
    mel._call(fn, "call", 1, 55, "c")
    mel._call(fn, "call", 0, 56, "d")
    assert log == [("a", 0, 100), ("b", 1, 101), ("c", 1, 55), ("d", 0, 56)] and now == [0]

"""Refusals of grouped routing, gradient clipping and the microscaled calls on the CPU: every call here
fails its argument checks, so no kernel is ever launched."""
import ctypes

import pytest

from test_abi_residual import at, desc, err, lib, params  # noqa: F401  (lib: fixture)

P = ctypes.c_void_p
BY = ctypes.byref


def router(T=64, E=32, k=4, score=1, groups=4, topk_groups=2, group_top=2, renorm=1, scale=2.5):
    from mixture_experts_lora_amd._lib import MoeGroupedRouter
    return MoeGroupedRouter(T, E, k, score, groups, topk_groups, group_top, renorm, scale)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(E=0), 1), (dict(E=1028), 1), (dict(k=0), 1), (dict(k=33, groups=1, topk_groups=1), 1),
    (dict(E=64, k=33, groups=1, topk_groups=1), 2), (dict(score=2), 1), (dict(score=-1), 1),
    (dict(groups=0), 1), (dict(groups=5), 1), (dict(E=65, groups=65), 2), (dict(topk_groups=0), 1),
    (dict(topk_groups=5), 1), (dict(k=9, topk_groups=1), 1), (dict(group_top=0), 1),
    (dict(group_top=3), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(T=1 << 30, k=2), 1),
])
def test_router(lib, kw, status):  # noqa: F811
    r = router(**kw)
    assert lib.moe_route_grouped(BY(r), at(0), at(1), at(2), at(3), None) == status
    assert err(lib)
    assert lib.moe_route_grouped_bwd(BY(r), at(0), at(1), at(2), at(3), None) == status


def test_route_buffers(lib):  # noqa: F811
    r = router()
    ok = [at(0), at(1), at(2), at(3)]  # logits, bias, topk_ids, topk_w
    for i in (0, 2, 3):
        a = list(ok)
        a[i] = None
        assert lib.moe_route_grouped(BY(r), *a, None) == 1 and "null" in err(lib)
    for i, other in ((2, 0), (3, 0), (2, 1), (3, 2)):
        a = list(ok)
        a[i] = P(a[other].value + 4)
        assert lib.moe_route_grouped(BY(r), *a, None) == 1 and "overlaps" in err(lib)
    assert lib.moe_route_grouped(None, *ok, None) == 1
    for i in range(4):  # logits, topk_ids, d_topk_w, d_logits
        a = list(ok)
        a[i] = None
        assert lib.moe_route_grouped_bwd(BY(r), *a, None) == 1 and "null" in err(lib)
    for i in range(3):
        a = list(ok)
        a[3] = a[i]
        assert lib.moe_route_grouped_bwd(BY(r), *a, None) == 1 and "overlaps" in err(lib)


def grads(*items):
    """(count, array) of (src, dst, n, dtype); addresses as numbers."""
    from mixture_experts_lora_amd._lib import MoeGrad
    return len(items), (MoeGrad * max(len(items), 1))(*(MoeGrad(*i) for i in items))


A, B = 0x10000000, 0x20000000


@pytest.mark.parametrize("bad", [(A, A, 8, 3), (A, A, -1, 0), (A, A, (1 << 40) + 1, 0), (None, A, 8, 0),
                                 (A + 2, A, 8, 0), (A + 1, A, 8, 1)], ids=str)
def test_gradient_lists(lib, bad):  # noqa: F811
    n = ctypes.c_size_t()
    g = grads((B, B, 64, 0), bad)
    assert lib.moe_grad_norm_workspace_bytes(*g, BY(n)) == 1 and "gradient 1" in err(lib)
    assert lib.moe_grad_norm(*g, at(3), at(4), 1 << 20, None) == 1
    assert lib.moe_grad_clip(*g, at(3), 1.0, 1e-6, None) == 1


def test_gradient_calls(lib):  # noqa: F811
    n = ctypes.c_size_t()
    g = grads((A, A, 1 << 20, 0), (B, B, 64, 1))
    assert lib.moe_grad_norm_workspace_bytes(-1, g[1], BY(n)) == 1
    assert lib.moe_grad_norm_workspace_bytes((1 << 20) + 1, g[1], BY(n)) == 2
    assert lib.moe_grad_norm_workspace_bytes(2, None, BY(n)) == 1
    assert lib.moe_grad_norm_workspace_bytes(*g, None) == 1
    assert lib.moe_grad_norm_workspace_bytes(*g, BY(n)) == 0 and n.value > 0
    need = n.value
    norm, ws = 0x30000000, 0x40000000
    assert lib.moe_grad_norm(*g, None, ws, need, None) == 1
    assert lib.moe_grad_norm(*g, norm, None, need, None) == 1
    assert lib.moe_grad_norm(*g, norm, ws, need - 1, None) == 3
    assert lib.moe_grad_norm(*g, norm + 2, ws, need, None) == 1
    assert lib.moe_grad_norm(*g, norm, ws + 8, need, None) == 1
    assert lib.moe_grad_norm(*g, A + 64, ws, need, None) == 1 and "overlaps" in err(lib)
    assert lib.moe_grad_norm(*g, norm, B, need, None) == 1 and "overlaps" in err(lib)
    assert lib.moe_grad_norm(*g, ws, ws, need, None) == 1 and "overlaps" in err(lib)
    for most, eps in ((-1.0, 1e-6), (float("nan"), 1e-6), (float("inf"), 1e-6), (1.0, 0.0),
                      (1.0, -1.0), (1.0, float("nan")), (1.0, float("inf"))):
        assert lib.moe_grad_clip(*g, norm, most, eps, None) == 1
    assert lib.moe_grad_clip(*g, None, 1.0, 1e-6, None) == 1
    assert lib.moe_grad_clip(*g, norm + 1, 1.0, 1e-6, None) == 1
    for items in ([(A, None, 8, 0)], [(A, B + 2, 8, 0)], [(A, A + 4, 8, 0)], [(A, A, 8, 0), (A, A, 8, 0)],
                  [(A, B, 8, 0), (A + 64, B + 16, 8, 0)], [(A, B, 8, 0), (B + 16, B + 64, 8, 0)],
                  [(A, norm - 8, 8, 1)]):
        assert lib.moe_grad_clip(*grads(*items), norm, 1.0, 1e-6, None) == 1, items


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), 1), (dict(fmt=-1), 1), (dict(dtype=3), 1), (dict(rows=-1), 1), (dict(cols=0), 2),
    (dict(cols=48), 2), (dict(cols=-32), 2), (dict(rows=1 << 29), 1), (dict(src=None), 1),
    (dict(codes=None), 1), (dict(scales=None), 1), (dict(src=A + 8), 1), (dict(codes=B + 4), 1),
    (dict(scales=0x30000001), 1), (dict(codes=A + 16), 1), (dict(scales=A + 160), 1), (dict(scales=B), 1),
])
def test_mx_formats(lib, kw, status):  # noqa: F811
    v = dict(fmt=0, dtype=1, rows=64, cols=128, src=A, codes=B, scales=0x30000000)
    v.update(kw)
    assert lib.moe_mx_quantize(*v.values(), None) == status and err(lib)
    if v["scales"] != v["codes"]:  # both are read here
        a = (v["fmt"], v["dtype"], v["rows"], v["cols"], v["codes"], v["scales"], v["src"], None)
        assert lib.moe_mx_dequantize(*a) == status


def test_mx_nothing_to_do(lib):  # noqa: F811
    assert lib.moe_mx_quantize(0, 1, 0, 128, None, None, None, None) == 0
    assert lib.moe_mx_dequantize(1, 0, 0, 128, None, None, None, None) == 0
    assert [lib.moe_mx_scale_cols(c) for c in (0, 32, 512, 544, 2880)] == [0, 16, 16, 32, 96]


def shape(T=8, K=64, N=32, E=4, k=2, a_format=0, gather=1, swiglu=1, out=3):
    from mixture_experts_lora_amd._lib import MoeMxLinearShape
    return MoeMxLinearShape(T, K, N, E, k, a_format, gather, swiglu, out)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(k=0), 1), (dict(E=-1), 1), (dict(E=1025), 1),
    (dict(k=5), 1), (dict(E=64, k=33), 1), (dict(E=0, k=1), 1), (dict(E=0, k=2, gather=0), 1),
    (dict(a_format=2), 1), (dict(out=0), 1), (dict(out=4), 1), (dict(K=48), 2), (dict(N=40), 2),
    (dict(N=12, out=1), 2), (dict(K=(1 << 20) + 32, N=32), 2), (dict(N=(1 << 20) + 32, K=32), 2),
    (dict(T=1 << 30), 1), (dict(T=1 << 28, K=128), 1), (dict(K=1 << 16, N=1 << 15), 1),
    (dict(T=1 << 20, K=2048), 1),
])
def test_mx_linear_shapes(lib, kw, status):  # noqa: F811
    n = ctypes.c_size_t()
    s = shape(**kw)
    assert lib.moe_mx_linear_workspace_bytes(BY(s), BY(n)) == status and err(lib)
    a = [at(i) for i in range(8)]
    assert lib.moe_mx_linear(BY(s), *a, None, 0, None) == status


def test_mx_linear_buffers(lib):  # noqa: F811
    n = ctypes.c_size_t()
    s = shape()
    assert lib.moe_mx_linear_workspace_bytes(BY(s), BY(n)) == 0
    assert lib.moe_mx_linear_workspace_bytes(BY(s), None) == 1
    assert lib.moe_mx_linear_workspace_bytes(None, BY(n)) == 1
    names = ("a", "a_scales", "rows", "offsets", "w", "w_scales", "y", "y_scales")
    ok = [at(i) for i in range(8)]

    def call(sh=s, **kw):
        a = dict(zip(names, ok))
        a.update(kw)
        return lib.moe_mx_linear(BY(sh), *(a[x] for x in names), None, 0, None)

    for i, x in enumerate(names):
        assert call(**{x: None}) == 1 and "null" in err(lib)
        assert call(**{x: P(ok[i].value + 2)}) == 1 and "boundary" in err(lib)
        if x not in ("y", "y_scales"):
            assert call(y=ok[i]) == 1 and "overlaps" in err(lib)
            assert call(y_scales=ok[i]) == 1 and "overlaps" in err(lib)
    assert call(y=ok[7]) == 1
    plain = shape(out=1, N=64)
    assert call(plain) == 1 and "y_scales" in err(lib)
    # a 16-bit result reaches twice as far
    assert call(plain, y_scales=None, y=P(ok[0].value - 16 * 64 * 2 + 16)) == 1 and "overlaps" in err(lib)


def test_residual_norm_mx(lib):  # noqa: F811
    names = ("h", "y", "params", "rng", "site", "h_out", "x_out", "x_codes", "x_scales", "stats")
    q = params()
    ok = (at(0), at(1), BY(q), None, 0, at(2), at(3), at(4), at(5), at(6))

    def call(d, **kw):
        a = dict(zip(names, ok))
        a.update(kw)
        return lib.moe_residual_norm_mx_fwd(BY(d), *(a[n] for n in names), None)

    d = desc(H=128, pre=1)
    assert call(desc(pre=0)) == 1 and "pre norm" in err(lib)
    assert call(desc(H=136)) == 2 and "32" in err(lib)
    assert call(desc(T=0)) == 1
    for n in ("x_codes", "x_scales", "h_out"):
        assert call(d, **{n: None}) == 1
    for n in ("h", "y", "h_out", "x_out", "x_codes", "x_scales", "stats"):
        v = dict(zip(names, ok))[n]
        assert call(d, **{n: P(v.value + 4)}) == 1 and "boundary" in err(lib)
    for n in ("h", "y", "h_out", "x_out", "stats"):
        v = dict(zip(names, ok))[n]
        assert call(d, x_codes=v) == 1 and "overlaps" in err(lib)
        assert call(d, x_scales=v) == 1 and "overlaps" in err(lib)
    assert call(d, x_codes=at(5)) == 1 and "overlaps" in err(lib)

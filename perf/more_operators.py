"""Measured cases of routing with groups and a bias, of microscaled formats, and of gradient clipping.

- route: top-k experts by softmax or sigmoid scores plus a bias for balance, the best groups of
  experts first; weights renormalised and scaled. With its backward.
- quantize: rows to E2M1 (4 bits) or E4M3 (8 bits) with one power-of-two scale per 32, and back.
- product: y = a w^T of microscaled operands, one weight matrix or one per expert, optionally
  with SwiGLU and an 8-bit result.
- norm: the residual's addition and an RMS norm, its output in 8 bits with scales.
- clip: the norm of all gradients together, and the gradients scaled to at most a given one.

With own = False, run() computes them from elementary torch operations in 32 bits; scores that
decide a choice, and sums of squares over many tensors, in 64.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ cases
def _route(name, T, E, k, bwd, score="sigmoid", groups=1, topk_groups=1, group_top=2, renorm=True,
           scale=1.0, bias=True):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "bwd": bwd, "score": score,
            "groups": groups, "topk_groups": topk_groups, "group_top": group_top,
            "renorm": renorm, "scale": scale, "bias": bias}


def _quantize(name, rows, cols, dtype, fmt):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype, "fmt": fmt}


def _product(name, T, K, N, fmt, out, E=0, k=1, act="none", gather=False):
    """E = 0: one weight matrix. Otherwise T * k rows over E experts; gather: rows of T tokens."""
    return {"name": name, "op": "product", "T": T, "K": K, "N": N, "fmt": fmt, "out": out, "E": E,
            "k": k, "act": act, "gather": gather}


def _norm(name, T, H, dtype, post="none", alpha=1.0, shift=0.0):
    return {"name": name, "op": "norm", "T": T, "H": H, "dtype": dtype, "post": post,
            "alpha": alpha, "shift": shift}


def _clip(name, layers, E, H, I, r, dtype):
    return {"name": name, "op": "clip", "layers": layers, "E": E, "H": H, "I": I, "r": r,
            "dtype": dtype}


def listed():
    return [
        # one decoded token through a router of 256 experts in 8 groups
        _route("route_token", 1, 256, 8, False, groups=8, topk_groups=4, scale=2.5),
        # the same router over a training step, and its backward
        _route("route_train", 8192, 256, 8, False, groups=8, topk_groups=4, scale=2.5),
        _route("route_bwd_train", 16384, 128, 8, True, score="softmax", scale=1.0),
        # activations of a small batch to 8 bits, and a layer's gate_up weights to 4 bits
        _quantize("quantize_small", 300, 608, "f16", "fp8"),
        _quantize("quantize_weights", 32 * 5760, 2880, "bf16", "fp4"),
        # one decoded token through its experts' gate and up projections
        _product("product_token", 1, 2880, 2880, "fp8", "bf16", E=32, k=4, act="swiglu", gather=True),
        # the same projections over a training step's tokens, the result in 8 bits for the next
        _product("product_experts", 8192, 2880, 2880, "fp8", "mx8", E=32, k=4, act="swiglu", gather=True),
        # a dense projection, both operands in 4 bits
        _product("product_dense", 8192, 4096, 2880, "fp4", "bf16"),
        # one decoded token, and a training step on wide rows with a norm after the block too
        _norm("norm_token", 1, 2880, "bf16"),
        _norm("norm_train", 8192, 7168, "bf16", post="rms", alpha=0.5, shift=1.0),
        # the adapters of a small float32 layer, and of twelve large layers
        _clip("clip_small", 1, 8, 256, 128, 8, "f32"),
        _clip("clip_train", 12, 32, 2880, 2880, 16, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["route", "route", "quantize", "product", "product", "norm", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if kind == "route":
        groups = rng.choice([1, 2, 4, 8])
        E = groups * _log(rng, 4, 512 // groups)
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(32, E // groups * topk_groups))
        case = _route("", _log(rng, 1, 16384), E, k, rng.random() < 0.5,
                      rng.choice(["softmax", "sigmoid"]), groups, topk_groups, rng.choice([1, 2]),
                      rng.random() < 0.6, rng.choice([1.0, 2.5, 16.0]), rng.random() < 0.7)
    elif kind == "quantize":
        cols = 32 * _log(rng, 1, 512)
        rows = min(_log(rng, 1, 200000), 32 * 5760 * 2880 // cols)
        case = _quantize("", rows, cols, dtype, rng.choice(["fp4", "fp8"]))
    elif kind == "product":
        K, act = 32 * _log(rng, 2, 224), rng.choice(["none", "swiglu"])
        out = rng.choice(["bf16", "f16", "mx8"])
        N = 32 * _log(rng, 1, 180) if out == "mx8" else 8 * _log(rng, 2, 720)
        E = rng.choice([0, 0, 4, 8, 32, 100])
        E = min(E, 32 * 5760 * 2880 // (K * N)) if E else 0
        k = min(rng.choice([1, 2, 4]), max(E, 1))
        T = min(_log(rng, 1, 16384), 32768 * 2880 * 5760 // (2 * K * N * k))
        case = _product("", T, K, N, rng.choice(["fp4", "fp8"]), out, E, k, act,
                        E > 0 and rng.random() < 0.5)
    elif kind == "norm":
        H = 32 * _log(rng, 2, 224)
        T = min(_log(rng, 1, 32768), 8192 * 7168 // H)
        case = _norm("", T, H, dtype, rng.choice(["none", "rms"]), rng.choice([1.0, 0.5, 0.22]),
                     rng.choice([0.0, 1.0]))
    else:
        H, I, r = 8 * _log(rng, 4, 360), 8 * _log(rng, 4, 360), rng.choice([4, 8, 12, 16])
        case = _clip("", rng.randint(1, 12), rng.choice([1, 3, 8, 32]), H, I, r, dtype)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": case, "gen": g}
    {"route": _prepare_route, "quantize": _prepare_quantize, "product": _prepare_product,
     "norm": _prepare_norm, "clip": _prepare_clip}[case["op"]](case, s, normal)
    del s["gen"]
    return s


def _prepare_route(case, s, normal):
    T, E, k = case["T"], case["E"], case["k"]
    s["logits"] = normal(T, E)
    s["bias"] = normal(E, std=0.05) if case["bias"] else None
    s["ids"] = torch.empty(T, k, device="cuda", dtype=torch.int32)
    s["w"] = torch.empty(T, k, device="cuda")
    if case["bwd"]:  # the forward's choice, and the gradient that arrives at the weights
        s["ids"] = _choose(s["logits"], s["bias"], case).int()
        s["dw"] = normal(T, k)
        s["dlogits"] = torch.empty_like(s["logits"])
    if own:
        import mixture_experts_lora_amd as mel
        s["router"] = mel.GroupedRouter(E, k, score=case["score"], groups=case["groups"],
                                        topk_groups=case["topk_groups"],
                                        group_top=case["group_top"], renorm=case["renorm"],
                                        scale=case["scale"])


def _blank(rows, cols, fmt):
    codes = torch.empty(rows, cols // 2 if fmt == "fp4" else cols, device="cuda", dtype=torch.uint8)
    return codes, torch.empty(rows, _scale_cols(cols), device="cuda", dtype=torch.uint8)


def _prepare_quantize(case, s, normal):
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    # weights, whose channels differ in size
    s["x"] = (normal(rows, cols) * normal(1, cols).exp() * cols ** -0.5).to(dt)
    s["codes"], s["scales"] = _blank(rows, cols, case["fmt"])
    s["back"] = torch.empty_like(s["x"])


def _coded(x, fmt):
    """Codes and scales of x as the products take them: two 4-bit codes a byte, low first."""
    v, e = _mx(x, fmt)
    if fmt == "fp8":
        codes = v.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        m = v.abs()
        c = torch.where(m < 2.0, m * 2.0, torch.where(m < 4.0, m + 2.0, m * 0.5 + 4.0)).to(torch.uint8)
        c = c + 8 * torch.signbit(v).to(torch.uint8)
        codes = c[..., 0::2] + 16 * c[..., 1::2]
    scales = torch.zeros(*x.shape[:-1], _scale_cols(x.shape[-1]), device=x.device, dtype=torch.uint8)
    scales[..., :e.shape[-1]] = (e + 127).to(torch.uint8)
    return codes.contiguous(), scales


def _prepare_product(case, s, normal):
    T, K, N, E, k = case["T"], case["K"], case["N"], case["E"], case["k"]
    M, n_w = T * k, N * (2 if case["act"] == "swiglu" else 1)
    s["a"], s["a_scales"] = _coded(normal(T if case["gather"] else M, K), case["fmt"])
    per = [_coded(normal(n_w, K, std=K ** -0.5), "fp4") for _ in range(max(E, 1))]
    s["w"], s["w_scales"] = (torch.stack([p[i] for p in per]) if E else per[0][i] for i in range(2))
    del per
    s["rows"] = s["offsets"] = None
    if E:  # tokens spread over the experts, some more popular than others
        score = torch.rand(T, E, generator=s["gen"], device="cuda").log().neg()
        score = score / torch.linspace(1.0, 2.0, E, device="cuda")
        pairs = score.argsort(1)[:, :k].reshape(-1)
        counts = (pairs[:, None] == torch.arange(E, device="cuda")).sum(0)
        s["offsets"] = torch.zeros(E + 1, device="cuda", dtype=torch.int32)
        s["offsets"][1:] = counts.cumsum(0)
        order = pairs.argsort(stable=True)
        s["expert"] = pairs[order]
        s["rows"] = order.int() if case["gather"] else None
        s["most"] = int(counts.max())
    if case["out"] == "mx8":
        s["y"], s["y_scales"] = _blank(M, N, "fp8")
    else:
        s["y"], s["y_scales"] = torch.empty(M, N, device="cuda", dtype=DTYPES[case["out"]]), None
    if own:
        import mixture_experts_lora_amd as mel
        s["shape"] = mel.MXLinear(T, K, N, a_format=case["fmt"], out=case["out"], act=case["act"],
                                  E=E, k=k, gather=case["gather"])
        s["ws"] = torch.empty(max(1, mel.moe_mx_linear_workspace_bytes(s["shape"])), device="cuda",
                              dtype=torch.uint8)


def _prepare_norm(case, s, normal):
    T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
    s["params"] = {"w_pre": normal(H, std=0.1, mean=1.0 - case["shift"], dtype=dt)}
    if case["post"] != "none":
        s["params"]["w_post"] = normal(H, std=0.1, mean=1.0 - case["shift"], dtype=dt)
    # a stream that has grown over the layers, and a block's output
    s["h"], s["y"] = normal(T, H, std=2.0, dtype=dt), normal(T, H, dtype=dt)
    s["h_out"] = torch.empty_like(s["h"])
    s["codes"], s["scales"] = _blank(T, H, "fp8")
    s["stats"] = torch.zeros(T, 4, device="cuda")
    if own:
        import mixture_experts_lora_amd as mel
        s["desc"] = mel.Residual(T, H, case["dtype"], post=case["post"], pre="rms",
                                 alpha=case["alpha"], weight_shift=case["shift"], eps=EPS)


def _prepare_clip(case, s, normal):
    E, H, I, r, dt = case["E"], case["H"], case["I"], case["r"], DTYPES[case["dtype"]]
    shapes = [(E, r, H), (E, 2 * I, r), (E, r, I), (E, H, r)] * case["layers"]
    s["grads"] = [normal(*d, std=1e-3, dtype=dt) for d in shapes]
    s["out"] = [torch.empty_like(g) for g in s["grads"]]
    s["norm"] = torch.empty(1, device="cuda")
    s["max_norm"] = 0.37e-3 * math.sqrt(sum(g.numel() for g in s["grads"]))
    if own:
        import mixture_experts_lora_amd as mel
        s["list"] = mel.GradList(s["grads"], out=s["out"])
        s["ws"] = torch.empty(max(1, mel.moe_grad_norm_workspace_bytes(s["list"])), device="cuda",
                              dtype=torch.uint8)


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "quantize": _plain_quantize, "product": _plain_product,
            "norm": _plain_norm, "clip": _plain_clip}[state["case"]["op"]](state)


def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn)


def _e8m0(scales):
    return scales.view(torch.float8_e8m0fnu)


def _run_own(s):
    import mixture_experts_lora_amd as mel
    case = s["case"]
    if case["op"] == "route":
        if case["bwd"]:
            mel.moe_route_grouped_bwd(s["router"], s["logits"], s["ids"], s["dw"], s["dlogits"])
            return {"dlogits": s["dlogits"]}
        mel.moe_route_grouped(s["router"], s["logits"], s["ids"], s["w"], bias=s["bias"])
        return {"ids": s["ids"], "w": s["w"]}
    if case["op"] == "quantize":
        mel.moe_mx_quantize(s["x"], s["codes"], s["scales"], case["fmt"])
        mel.moe_mx_dequantize(s["codes"], s["scales"], s["back"], case["fmt"])
        return {"values": s["back"], "scales": _e8m0(s["scales"])}
    if case["op"] == "product":
        mel.moe_mx_linear(s["shape"], s["a"], s["a_scales"], s["w"], s["w_scales"], s["y"], s["ws"],
                          y_scales=s["y_scales"], rows=s["rows"], offsets=s["offsets"])
        if case["out"] == "mx8":
            return {"codes": _e4m3(s["y"]), "scales": _e8m0(s["y_scales"])}
        return {"y": s["y"]}
    if case["op"] == "norm":
        mel.moe_residual_norm_mx_fwd(s["desc"], s["h"], s["y"], s["params"], s["h_out"],
                                     s["codes"], s["scales"], s["stats"])
        return {"h_out": s["h_out"], "codes": _e4m3(s["codes"]), "scales": _e8m0(s["scales"]),
                "stats": s["stats"]}
    mel.moe_grad_norm(s["list"], s["norm"], s["ws"])
    mel.moe_grad_clip(s["list"], s["norm"], s["max_norm"])
    return {"norm": s["norm"], "grads": s["out"]}


# ---- route
def _choose(logits, bias, case):
    """[T, k] experts: the best scores + bias within the best groups, ties to the lowest index."""
    T, E = logits.shape
    v = logits.double()
    if case["score"] == "sigmoid":
        v = 1.0 / (1.0 + torch.exp(-v))
    else:
        v = torch.exp(v - v.amax(1, keepdim=True))
        v = v / v.sum(1, keepdim=True)
    if bias is not None:
        v = v + bias.double()
    G = case["groups"]
    if G > 1:
        grouped = v.view(T, G, E // G)
        best = grouped.sort(dim=2, descending=True).values[:, :, :min(case["group_top"], E // G)].sum(2)
        keep = best.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        mask = torch.zeros(T, G, device=v.device, dtype=torch.bool).scatter_(1, keep, True)
        v = torch.where(mask[:, :, None], grouped, -math.inf).view(T, E)
    return v.sort(dim=1, descending=True, stable=True).indices[:, :case["k"]]


def _plain_route(s):
    case, logits = s["case"], s["logits"]
    ids = s["ids"].long() if case["bwd"] else _choose(logits, s["bias"], case)
    c = case["scale"]
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-logits))
    else:
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    chosen = p.gather(1, ids)
    total = chosen.sum(1, keepdim=True) if case["renorm"] else torch.ones_like(chosen[:, :1])
    if not case["bwd"]:
        return {"ids": ids.int(), "w": c * chosen / total}
    dp = c * s["dw"] / total  # the gradient at the chosen scores
    if case["renorm"]:
        dp = dp - (dp * chosen).sum(1, keepdim=True) / total
    d = torch.zeros_like(logits).scatter_(1, ids, dp)
    if case["score"] == "sigmoid":
        d = d * p * (1.0 / (1.0 + torch.exp(logits)))
    else:
        d = p * (d - (d * p).sum(1, keepdim=True))
    return {"dlogits": d}


# ---- microscaled formats: an element is v * 2^e, e one number per 32 elements
def _scale_cols(cols):
    return 16 * ((cols + 511) // 512)


def _mx(x, fmt):
    """The elements' values v (float32) and the exponents e of x's blocks."""
    b = x.float().unflatten(-1, (-1, 32))
    top, bits, least, most = (2, 1, 0, 6.0) if fmt == "fp4" else (8, 3, -6, 448.0)
    e = (torch.frexp(b.abs().amax(-1)).exponent - 1 - top).clamp(min=-127)
    e = torch.where(b.abs().amax(-1) > 0, e, -127)
    v = torch.ldexp(b, -e[..., None])
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v).exponent - 1).clamp(min=least) - bits)
    v = ((v / step).round() * step).clamp(-most, most)
    return v.flatten(-2), e


def _packed_scales(e, cols):
    """Exponents as [.., scale_cols] scales; those past the row's blocks have the code 0."""
    out = torch.zeros(*e.shape[:-1], _scale_cols(cols), device=e.device, dtype=torch.uint8)
    out[..., :e.shape[-1]] = (e + 127).to(torch.uint8)
    return _e8m0(out)


def _plain_quantize(s):
    x = s["x"]
    v, e = _mx(x, s["case"]["fmt"])
    back = torch.ldexp(v.unflatten(-1, (-1, 32)), e[..., None]).flatten(-2)
    return {"values": back.to(x.dtype), "scales": _packed_scales(e, x.shape[-1])}


def _values(codes, scales, fmt):
    """float32 values of codes [.., K] (K / 2 bytes in 4 bits) with their scales."""
    if fmt == "fp8":
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
        table = torch.cat([table, -table])
        v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    v = v.unflatten(-1, (-1, 32))
    return (v * torch.exp2(scales[..., :v.shape[-2]].float() - 127.0)[..., None]).flatten(-2)


def _plain_product(s):
    case = s["case"]
    E, k, M = case["E"], case["k"], case["T"] * case["k"]
    a = _values(s["a"], s["a_scales"], case["fmt"])
    if case["gather"]:
        a = a[s["rows"].long() // k]
    if not E:
        z = a @ _values(s["w"], s["w_scales"], "fp4").t()
    elif M <= min(E, 16):  # few rows: each row's own matrix
        w = _values(s["w"][s["expert"]], s["w_scales"][s["expert"]], "fp4")
        z = (w * a[:, None, :]).sum(2)
    else:  # each expert's rows, filled up to the most that one has
        place = torch.arange(M, device=a.device) - s["offsets"].long()[s["expert"]]
        full = torch.zeros(E, s["most"], a.shape[1], device=a.device)
        full[s["expert"], place] = a
        w = _values(s["w"], s["w_scales"], "fp4").transpose(1, 2).contiguous()
        z = torch.bmm(full, w)[s["expert"], place]
    if case["act"] == "swiglu":
        gate, up = z[:, :case["N"]], z[:, case["N"]:]
        z = gate / (1.0 + torch.exp(-gate)) * up
    if case["out"] != "mx8":
        return {"y": z.to(DTYPES[case["out"]])}
    v, e = _mx(z, "fp8")
    return {"codes": v.to(torch.float8_e4m3fn), "scales": _packed_scales(e, case["N"])}


# ---- norm
def _rms(t, w, shift):
    rstd = (t.square().mean(1, keepdim=True) + EPS).rsqrt()
    return t * rstd * (shift + w.float()), rstd


def _plain_norm(s):
    case, prm, dt = s["case"], s["params"], s["h"].dtype
    stats = torch.zeros_like(s["stats"])
    v = s["y"].float()
    if case["post"] != "none":
        v, stats[:, 1:2] = _rms(v, prm["w_post"], case["shift"])
    h_out = (s["h"].float() + case["alpha"] * v).to(dt)
    # the norm of the stream as it is stored, in the layer's type, and from there in 8 bits
    x, stats[:, 3:4] = _rms(h_out.float(), prm["w_pre"], case["shift"])
    q, e = _mx(x.to(dt), "fp8")
    return {"h_out": h_out, "codes": q.to(torch.float8_e4m3fn),
            "scales": _packed_scales(e, case["H"]), "stats": stats}


# ---- clip
def _plain_clip(s):
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
    c = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return {"norm": norm.float().view(1), "grads": [(g.float() * c).to(g.dtype) for g in s["grads"]]}


# ------------------------------------------------------------------ what a pass needs
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        if case["bwd"]:
            return {"bytes": 4 * T * (2 * E + 2 * k), "flops": 10 * T * E}
        return {"bytes": 4 * (T * (E + 2 * k) + E * case["bias"]), "flops": 10 * T * E}
    es = 4 if case.get("dtype") == "f32" else 2
    if op == "quantize":  # to codes and scales, and back from them
        n = case["rows"] * case["cols"]
        coded = n * (0.5 if case["fmt"] == "fp4" else 1.0) + case["rows"] * _scale_cols(case["cols"])
        return {"bytes": 2 * n * es + 2 * coded, "flops": 6 * n}
    if op == "product":
        T, K, N, E, M = case["T"], case["K"], case["N"], case["E"], case["T"] * case["k"]
        n_w = N * (2 if case["act"] == "swiglu" else 1)
        a_rows = T if case["gather"] else M
        a = a_rows * (K * (0.5 if case["fmt"] == "fp4" else 1.0) + _scale_cols(K))
        w = n_w * (K * 0.5 + _scale_cols(K)) * max(1, min(E, M))
        y = M * (N + _scale_cols(N) if case["out"] == "mx8" else 2 * N)
        return {"bytes": a + w + y + 4 * (E + 1) * (E > 0) + 4 * M * case["gather"],
                "flops": 2 * M * n_w * K}
    if op == "norm":
        T, H = case["T"], case["H"]
        vec = H * es * (1 + (case["post"] != "none"))
        return {"bytes": T * (3 * H * es + H + _scale_cols(H) + 16) + vec, "flops": 14 * T * H}
    n = case["layers"] * case["E"] * case["r"] * (2 * case["H"] + 3 * case["I"])
    return {"bytes": 3 * n * es, "flops": 3 * n}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "quantize": _exact_quantize, "product": _exact_product,
            "norm": _exact_norm, "clip": _exact_clip}[case["op"]](case, s)


def _exact_route(case, s):
    l = s["logits"].double()
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    if case["bwd"]:  # the derivative of the weights, differentiated
        with torch.enable_grad():
            l.requires_grad_(True)
            p = (torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1))
            p = p.gather(1, s["ids"].long())
            w = p / p.sum(1, keepdim=True) if case["renorm"] else p
            grad, = torch.autograd.grad((case["scale"] * w * s["dw"].double()).sum(), l)
        return {"dlogits": grad}
    free = score + (0.0 if s["bias"] is None else s["bias"].double())
    if G > 1:  # take the best group again and again
        left = torch.stack([torch.topk(part, min(case["group_top"], E // G), 1).values.sum(1)
                            for part in free.chunk(G, 1)], 1)
        taken = torch.zeros(T, G, device=l.device, dtype=torch.bool)
        for _ in range(case["topk_groups"]):
            at = left.argmax(1, keepdim=True)
            taken.scatter_(1, at, True)
            left.scatter_(1, at, -math.inf)
        free = free.masked_fill(~taken.repeat_interleave(E // G, 1), -math.inf)
    ids = torch.empty(T, k, device=l.device, dtype=torch.int64)
    for j in range(k):
        ids[:, j] = free.argmax(1)
        free = free.scatter(1, ids[:, j:j + 1], -math.inf)
    p = score.gather(1, ids)
    w = case["scale"] * (p / p.sum(1, keepdim=True) if case["renorm"] else p)
    return {"ids": ids.int(), "w": w}


def _nearest64(x, fmt):
    """(values of the codes, exponents) of float64 rows: the nearest code, ties to an even one."""
    if fmt == "fp4":
        table = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        table = [m * 2.0 ** -9 for m in range(8)]
        table += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119]
    table = torch.tensor(table, device=x.device, dtype=torch.float64)
    top = math.floor(math.log2(table[-1].item()))
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - top, -127).clamp(min=-127)
    q = b * torch.exp2(-e.double())[..., None]
    mid = (table[1:] + table[:-1]) / 2
    lo = torch.searchsorted(mid, q.abs().contiguous())               # ties down
    hi = torch.searchsorted(mid, q.abs().contiguous(), right=True)   # ties up
    code = torch.where(lo % 2 == 0, lo, hi)
    return torch.copysign(table[code], q).flatten(-2), e


def _scales64(e, cols):
    out = torch.full((*e.shape[:-1], _scale_cols(cols)), 2.0 ** -127, device=e.device,
                     dtype=torch.float64)
    out[..., :e.shape[-1]] = torch.exp2(e.double())
    return out


def _exact_quantize(case, s):
    v, e = _nearest64(s["x"].double(), case["fmt"])
    back = (v.unflatten(-1, (-1, 32)) * torch.exp2(e.double())[..., None]).flatten(-2)
    return {"values": back, "scales": _scales64(e, case["cols"])}


def _decode64(codes, scales, fmt):
    if fmt == "fp8":
        c = codes.long()
        exp, man = (c >> 3) & 15, (c & 7).double()
        v = torch.where(exp > 0, (8 + man) * torch.exp2(exp.double() - 10), man * 2.0 ** -9)
        v = torch.where(c > 127, -v, v)
    else:
        c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
        exp, man = (c >> 1) & 3, (c & 1).double()
        v = torch.where(exp > 0, (2 + man) * torch.exp2(exp.double() - 2), man * 0.5)
        v = torch.where(c > 7, -v, v)
    e = scales[..., :v.shape[-1] // 32].repeat_interleave(32, -1)
    return v * torch.exp2(e.double() - 127)


def _exact_product(case, s):
    a = _decode64(s["a"], s["a_scales"], case["fmt"])
    if case["E"]:
        z = []
        bounds = s["offsets"].tolist()
        for e in range(case["E"]):
            lo, hi = bounds[e], bounds[e + 1]
            mine = a[torch.div(s["rows"][lo:hi].long(), case["k"], rounding_mode="floor")] \
                if case["gather"] else a[lo:hi]
            if hi > lo:
                z.append(torch.matmul(mine, _decode64(s["w"][e], s["w_scales"][e], "fp4").t()))
        z = torch.cat(z)
    else:
        z = torch.matmul(a, _decode64(s["w"], s["w_scales"], "fp4").t())
    if case["act"] == "swiglu":
        z = torch.nn.functional.silu(z[:, :case["N"]]) * z[:, case["N"]:]
    if case["out"] != "mx8":
        return {"y": z}
    v, e = _nearest64(z, "fp8")
    return {"codes": v, "scales": _scales64(e, case["N"])}


def _exact_norm(case, s):
    def norm(t, w):
        rstd = 1.0 / torch.sqrt((t * t).sum(1) / t.shape[1] + EPS)
        return t * rstd[:, None] * (w.double() + case["shift"]), rstd

    stats = torch.zeros(case["T"], 4, device="cuda", dtype=torch.float64)
    v = s["y"].double()
    if case["post"] != "none":
        v, stats[:, 1] = norm(v, s["params"]["w_post"])
    h = s["h"].double() + case["alpha"] * v
    x, stats[:, 3] = norm(h.to(s["h"].dtype).double(), s["params"]["w_pre"])
    q, e = _nearest64(x.to(s["h"].dtype).double(), "fp8")
    return {"h_out": h, "codes": q, "scales": _scales64(e, case["H"]), "stats": stats}


def _exact_clip(case, s):
    norm = sum((g.double() ** 2).sum() for g in s["grads"]) ** 0.5
    c = min(1.0, s["max_norm"] / (norm.item() + 1e-6))
    return {"norm": norm.reshape(1), "grads": [g.double() * c for g in s["grads"]]}

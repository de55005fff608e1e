"""Measured cases of the residual-stream operators around a MoE block.

Three operators, each with its backward:

- residual_norm: h' = h + alpha * g * dropout(post(y)) and x' = pre(h'), with post and pre
  an RMS norm, a layer norm or none, and g a gate per channel, per token or per element.
- dropout: y = keep ? x * scale : 0, the mask drawn from Philox4x32-10 at the element's index.
- linear: y = residual + dropout(act(x w^T + b)).

With own = False, run() computes them from elementary torch operations in 32 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------ cases
def _norm(name, T, H, dtype, bwd, post="none", pre="rms", gate="none", sigmoid=False, alpha=1.0,
          shift=0.0, p=0.0):
    return {"name": name, "op": "norm", "T": T, "H": H, "dtype": dtype, "bwd": bwd, "post": post,
            "pre": pre, "gate": gate, "sigmoid": sigmoid, "alpha": alpha, "shift": shift, "p": p}


def _dropout(name, T, H, dtype, p):
    return {"name": name, "op": "dropout", "T": T, "H": H, "dtype": dtype, "p": p}


def _linear(name, T, K, N, dtype, bwd, act="none", bias=True, residual=True, p=0.0):
    return {"name": name, "op": "linear", "T": T, "K": K, "N": N, "dtype": dtype, "bwd": bwd,
            "act": act, "bias": bias, "residual": residual, "p": p}


def listed():
    return [
        # one decoded token: add the block's output, norm for the next block
        _norm("norm_fwd_token", 1, 2880, "bf16", False),
        # the add and norm of an 8192-token training step, both directions
        _norm("norm_fwd_train", 8192, 2880, "bf16", False),
        _norm("norm_bwd_train", 8192, 2880, "bf16", True),
        # norms before and after the block, a gate per channel and dropout, on wide rows
        _norm("norm_fwd_sandwich", 16384, 2048, "f16", False, post="rms", gate="channel",
              alpha=0.5, shift=1.0, p=0.1),
        _norm("norm_bwd_sandwich", 8192, 7168, "bf16", True, post="rms", gate="channel",
              alpha=0.5, shift=1.0, p=0.1),
        # a small float32 layer with layer norms and a sigmoid gate per token
        _norm("norm_bwd_small", 333, 200, "f32", True, post="layer", pre="layer", gate="token",
              sigmoid=True),
        # activations of a small batch, and of a long context
        _dropout("dropout_small", 300, 584, "bf16", 0.1),
        _dropout("dropout_long", 65536, 2880, "bf16", 0.1),
        # one decoded token through an output projection into the residual stream
        _linear("linear_fwd_token", 1, 4096, 2880, "bf16", False),
        # the same projection over a training step, with dropout before the add
        _linear("linear_fwd_train", 8192, 4096, 2880, "bf16", False, p=0.1),
        # a ragged batch through an activation
        _linear("linear_fwd_ragged", 300, 584, 2048, "f16", False, act="silu", residual=False),
        # the backward of a projection with an activation, all three gradients
        _linear("linear_bwd_train", 8192, 2880, 2880, "bf16", True, act="gelu", residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    p = rng.choice([0.0, 0.05, 0.1, 0.25, 0.5])
    kind = rng.choice(["norm", "norm", "dropout", "linear", "linear"])
    if kind == "norm":
        H = 8 * _log(rng, 8, 896)
        T = min(_log(rng, 1, 32768), 8192 * 7168 // H)
        post = rng.choice(["none", "rms", "layer"])
        case = _norm("", T, H, dtype, rng.random() < 0.5, post, rng.choice(["none", "rms", "layer"]),
                     rng.choice(["none", "channel", "token", "full"]), rng.random() < 0.5,
                     rng.choice([1.0, 0.5, 0.22]), rng.choice([0.0, 1.0]), p)
    elif kind == "dropout":
        H = _log(rng, 64, 7168)
        case = _dropout("", min(_log(rng, 1, 65536), 65536 * 2880 // H), H, dtype, p)
    else:
        bwd = rng.random() < 0.5
        K, N = 8 * _log(rng, 8, 896), 8 * _log(rng, 8, 896)
        T = min(_log(rng, 1, 16384), 8192 * 2880 * 2880 // (K * N) + 1)
        case = _linear("", T, K, N, dtype, bwd, rng.choice(ACTS), rng.random() < 0.7,
                       not bwd and rng.random() < 0.5, p)
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dt)

    s = {"case": case, "dt": dt,
         "rng": torch.randint(0, 1 << 62, (2,), generator=g, device="cuda", dtype=torch.int64)}
    if case["op"] == "norm":
        _prepare_norm(case, s, normal)
    elif case["op"] == "dropout":
        s["x"] = normal(case["T"], case["H"])
        s["out"] = torch.empty_like(s["x"])
    else:
        _prepare_linear(case, s, normal)
    return s


def _prepare_norm(case, s, normal):
    T, H, dt = case["T"], case["H"], s["dt"]
    prm = {}
    for which in ("post", "pre"):
        if case[which] != "none":  # trained weights scatter around one
            prm["w_" + which] = normal(H, std=0.1, mean=1.0 - case["shift"])
        if case[which] == "layer":
            prm["b_" + which] = normal(H, std=0.1)
    if case["gate"] != "none":
        prm["gate"] = normal(*{"channel": (H,), "token": (T,), "full": (T, H)}[case["gate"]])
    # a stream that has grown over the layers, and a block's output
    s.update(params=prm, h=normal(T, H, std=2.0), y=normal(T, H))
    s["h_out"] = torch.empty_like(s["h"])
    s["x_out"] = torch.empty_like(s["h"]) if case["pre"] != "none" else None
    s["stats"] = torch.zeros(T, 4, device="cuda")
    if case["bwd"]:  # what the forward left, and the two gradients that arrive
        s["h_out"] = s.pop("h")
        for i, (which, t) in enumerate((("post", s["y"]), ("pre", s["h_out"]))):
            if case[which] != "none":
                mean, rstd = _stats(t.float(), case[which])
                s["stats"][:, 2 * i], s["stats"][:, 2 * i + 1] = mean[:, 0], rstd[:, 0]
        s["dh_out"] = normal(T, H)
        s["dx_out"] = normal(T, H) if case["pre"] != "none" else None
        s["dh"], s["dy"] = torch.empty_like(s["y"]), torch.empty_like(s["y"])
        s["grads"] = {"d" + n: torch.empty_like(t) for n, t in prm.items()}
    if own:
        import mixture_experts_lora_amd as mel
        s["desc"] = mel.Residual(T, H, case["dtype"], post=case["post"], pre=case["pre"],
                                 gate=case["gate"], gate_sigmoid=case["sigmoid"],
                                 alpha=case["alpha"], weight_shift=case["shift"], eps=EPS,
                                 dropout=case["p"])
        s["ws"] = torch.empty(max(1, mel.moe_residual_norm_workspace_bytes(s["desc"])),
                              device="cuda", dtype=torch.uint8)


def _prepare_linear(case, s, normal):
    T, K, N = case["T"], case["K"], case["N"]
    s["x"], s["w"] = normal(T, K), normal(N, K, std=K ** -0.5)
    s["b"] = normal(N, std=0.1) if case["bias"] else None
    if case["bwd"]:
        s["pre"] = None
        if case["act"] != "none":  # kept by the forward
            z = s["x"].float() @ s["w"].float().t()
            s["pre"] = (z if s["b"] is None else z + s["b"].float()).to(s["dt"])
        s["dout"] = normal(T, N)
        s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
        s["db"] = None if s["b"] is None else torch.empty_like(s["b"])
    else:
        s["res"] = normal(T, N) if case["residual"] else None
        s["out"] = torch.empty(T, N, device="cuda", dtype=s["dt"])
        s["pre"] = torch.empty_like(s["out"]) if case["act"] != "none" else None
    if own:
        import mixture_experts_lora_amd as mel
        s["shape"] = mel.LinearShape(T, K, N, case["dtype"], act=case["act"], dropout=case["p"])
        need = mel.moe_linear_workspace_bytes(s["shape"])[1 if case["bwd"] else 0]
        s["ws"] = torch.empty(max(1, need), device="cuda", dtype=torch.uint8)


EPS = 1e-5


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "norm":
        return _norm_bwd(state) if case["bwd"] else _norm_fwd(state)
    if case["op"] == "dropout":
        return _drop(state["x"].float(), state).to(state["dt"])
    return _linear_bwd(state) if case["bwd"] else _linear_fwd(state)


def _run_own(s):
    import mixture_experts_lora_amd as mel
    case = s["case"]
    if case["op"] == "norm" and not case["bwd"]:
        mel.moe_residual_norm_fwd(s["desc"], s["h"], s["y"], s["params"], s["h_out"], s["x_out"],
                                  s["stats"], rng=s["rng"])
        return {"h_out": s["h_out"], "x_out": s["x_out"], "stats": s["stats"]}
    if case["op"] == "norm":
        mel.moe_residual_norm_bwd(s["desc"], s["dh_out"], s["dx_out"], s["h_out"], s["y"],
                                  s["params"], s["stats"], s["dh"], s["dy"], s["grads"], s["ws"],
                                  rng=s["rng"])
        return {"dh": s["dh"], "dy": s["dy"], **s["grads"]}
    if case["op"] == "dropout":
        mel.moe_dropout(s["x"], s["out"], case["p"], rng=s["rng"])
        return s["out"]
    if not case["bwd"]:
        mel.moe_linear_fwd(s["shape"], s["x"], s["w"], s["out"], s["ws"], bias=s["b"],
                           residual=s["res"], pre=s["pre"], rng=s["rng"])
        return {"y": s["out"], "pre": s["pre"]}
    mel.moe_linear_bwd(s["shape"], s["dout"], s["x"], s["w"], s["pre"], s["dx"], s["dw"], s["db"],
                       s["ws"], rng=s["rng"])
    return {"dx": s["dx"], "dw": s["dw"], "dbias": s["db"]}


# ---- dropout: word i of counter c = element / 8 gives elements 2i (low half) and 2i + 1
M0, M1, W0, W1, LOW = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85, 0xFFFFFFFF


def _keep(n, p, rng, device):
    """[n] truth values: element i is kept."""
    c = torch.arange((n + 7) // 8, device=device)
    seed, off = rng[0], rng[1]
    k0, k1 = seed & LOW, (seed >> 32) & LOW
    x0, x1 = c & LOW, c >> 32
    x2, x3 = off & LOW, (off >> 32) & LOW
    for _ in range(10):  # the generator's rounds
        a, b = x0 * M0, x2 * M1  # low 64 bits of the product; the high word below
        x0, x1, x2, x3 = (((b >> 32) & LOW) ^ x1 ^ k0, b & LOW, ((a >> 32) & LOW) ^ x3 ^ k1, a & LOW)
        k0, k1 = (k0 + W0) & LOW, (k1 + W1) & LOW
    words = torch.stack([x0, x1, x2, x3], dim=-1)
    u16 = torch.stack([words & 0xFFFF, words >> 16], dim=-1).reshape(-1)[:n]
    return u16 >= int(p * 65536 + 0.5)


def _drop(v, s):
    """v (float32) with dropped elements 0 and kept ones scaled."""
    p = s["case"]["p"]
    if p == 0.0:
        return v
    keep = _keep(v.numel(), p, s["rng"], v.device).view(v.shape)
    scale = 65536.0 / (65536 - int(p * 65536 + 0.5))
    return torch.where(keep, v * scale, torch.zeros_like(v))


# ---- residual_norm
def _stats(t, kind):
    mean = t.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(t[:, :1])
    var = (t - mean).square().mean(1, keepdim=True)
    return mean, (var + EPS).rsqrt()


def _affine(xhat, prm, which, shift):
    v = xhat * (shift + prm["w_" + which].float())
    return v + prm["b_" + which].float() if "b_" + which in prm else v


def _gate(case, prm):
    if case["gate"] == "none":
        return 1.0
    g = prm["gate"].float()
    g = 1.0 / (1.0 + torch.exp(-g)) if case["sigmoid"] else g
    return g[:, None] if case["gate"] == "token" else g


def _norm_fwd(s):
    case, prm = s["case"], s["params"]
    stats = torch.zeros_like(s["stats"])
    v = s["y"].float()
    if case["post"] != "none":
        mean, rstd = _stats(v, case["post"])
        v = _affine((v - mean) * rstd, prm, "post", case["shift"])
        stats[:, 0:1], stats[:, 1:2] = mean, rstd
    h_out = (s["h"].float() + case["alpha"] * _gate(case, prm) * _drop(v, s)).to(s["dt"])
    x_out = None
    if case["pre"] != "none":  # the norm of the stream as it is stored
        t = h_out.float()
        mean, rstd = _stats(t, case["pre"])
        x_out = _affine((t - mean) * rstd, prm, "pre", case["shift"]).to(s["dt"])
        stats[:, 2:3], stats[:, 3:4] = mean, rstd
    return {"h_out": h_out, "x_out": x_out, "stats": stats}


def _norm_back(xhat, rstd, dv, w, kind):
    """Gradient at a norm's input from the gradient dv at its output."""
    d = dv * w
    c = (d * xhat).mean(1, keepdim=True)
    m = d.mean(1, keepdim=True) if kind == "layer" else 0.0
    return rstd * (d - m - xhat * c)


def _norm_bwd(s):
    case, prm, dt = s["case"], s["params"], s["dt"]
    mp, rp, mq, rq = (s["stats"][:, i:i + 1] for i in range(4))
    out = {}
    D = s["dh_out"].float()
    if case["pre"] != "none":
        xhat, dv = (s["h_out"].float() - mq) * rq, s["dx_out"].float()
        D = D + _norm_back(xhat, rq, dv, case["shift"] + prm["w_pre"].float(), case["pre"])
        out["dw_pre"] = (dv * xhat).sum(0).to(dt)
        if case["pre"] == "layer":
            out["db_pre"] = dv.sum(0).to(dt)
    out["dh"] = D.to(dt)
    v = s["y"].float()
    if case["post"] != "none":
        yhat = (v - mp) * rp
        v = _affine(yhat, prm, "post", case["shift"])
    g = _gate(case, prm)
    if case["gate"] != "none":
        dg = case["alpha"] * _drop(v, s) * D
        if case["gate"] != "full":
            dg = dg.sum(0 if case["gate"] == "channel" else 1)
        if case["sigmoid"]:
            gg = g.reshape(dg.shape)
            dg = dg * gg * (1.0 - gg)
        out["dgate"] = dg.to(dt)
    e = _drop(case["alpha"] * g * D, s)
    if case["post"] != "none":
        out["dw_post"] = (e * yhat).sum(0).to(dt)
        if case["post"] == "layer":
            out["db_post"] = e.sum(0).to(dt)
        e = _norm_back(yhat, rp, e, case["shift"] + prm["w_post"].float(), case["post"])
    out["dy"] = e.to(dt)
    return out


# ---- linear
def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _linear_fwd(s):
    case, dt = s["case"], s["dt"]
    z = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _drop(_act(z, case["act"]), s)
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(dt), "pre": z.to(dt) if case["act"] != "none" else None}


def _linear_bwd(s):
    case, dt = s["case"], s["dt"]
    dz = _drop(s["dout"].float(), s)
    if case["act"] != "none":
        dz = dz * _act_grad(s["pre"].float(), case["act"])
    return {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt),
            "dbias": None if s["b"] is None else dz.sum(0).to(dt)}


# ------------------------------------------------------------------ what a pass needs
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    T = case["T"]
    if case["op"] == "dropout":
        n = T * case["H"]
        return {"bytes": 2 * n * es, "flops": n}
    if case["op"] == "norm":
        H, pre = case["H"], case["pre"] != "none"
        vec = H * es * (sum(1 + (case[k] == "layer") for k in ("post", "pre") if case[k] != "none"))
        gate = es * {"none": 0, "channel": H, "token": T, "full": T * H}[case["gate"]]
        if not case["bwd"]:
            return {"bytes": T * H * es * (3 + pre) + vec + gate + 16 * T, "flops": 10 * T * H}
        reads = 1 + 2 * pre + (case["post"] != "none" or case["gate"] != "none")
        return {"bytes": T * H * es * (reads + 2) + 2 * (vec + gate) + 16 * T, "flops": 25 * T * H}
    K, N, act = case["K"], case["N"], case["act"] != "none"
    if not case["bwd"]:
        return {"bytes": es * (T * K + N * K + N * case["bias"] + T * N * (1 + act + case["residual"])),
                "flops": 2 * T * N * K}
    return {"bytes": es * (2 * T * K + 2 * N * K + N * case["bias"] + T * N * (1 + act)),
            "flops": 4 * T * N * K}


# ------------------------------------------------------------------ 64 bits
def _mul32(a, b):
    """High and low words of the product of two 32-bit values, from 16-bit halves."""
    al, ah, bl, bh = a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16
    mid = ah * bl + ((al * bl) >> 16)
    mid2 = al * bh + (mid & 0xFFFF)
    hi = ah * bh + (mid >> 16) + (mid2 >> 16)
    return hi, ((mid2 & 0xFFFF) << 16) | ((al * bl) & 0xFFFF)


def _mask64(shape, case, rng):
    """0 where dropped, 1 / P(keep) where kept."""
    n, t = math.prod(shape), round(case["p"] * 65536)
    seed, off = (int(v) for v in rng.tolist())
    idx = torch.arange((n + 7) // 8, device=rng.device)
    ctr = [idx % 2 ** 32, idx // 2 ** 32, torch.full_like(idx, off % 2 ** 32),
           torch.full_like(idx, off // 2 ** 32 % 2 ** 32)]
    key = [seed % 2 ** 32, seed // 2 ** 32 % 2 ** 32]
    for r in range(10):
        hi0, lo0 = _mul32(ctr[0], 0xD2511F53)
        hi1, lo1 = _mul32(ctr[2], 0xCD9E8D57)
        ctr = [hi1 ^ ctr[1] ^ key[0], lo1, hi0 ^ ctr[3] ^ key[1], lo0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    out = torch.empty(idx.numel(), 8, device=rng.device, dtype=torch.float64)
    for i in range(8):
        u = (ctr[i // 2] >> (16 * (i % 2))) % 65536
        out[:, i] = (u >= t).double() * (65536.0 / (65536 - t))
    return out.reshape(-1)[:n].reshape(shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        return s["x"].double() * _mask64(s["x"].shape, case, s["rng"])
    return _exact_norm(case, s) if case["op"] == "norm" else _exact_linear(case, s)


def _hat64(t, kind):
    """Normed rows, mean and 1 / deviation."""
    n = t.shape[1]
    mean = t.sum(1) / n if kind == "layer" else t.new_zeros(t.shape[0])
    c = t - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).sum(1) / n + EPS)
    return c * rstd[:, None], mean, rstd


def _exact_norm(case, s):
    d = {k: v.double() for k, v in s["params"].items()}
    T, H, shift, alpha = case["T"], case["H"], case["shift"], case["alpha"]
    y = s["y"].double()
    mask = _mask64((T, H), case, s["rng"])
    stats = torch.zeros(T, 4, device=y.device, dtype=torch.float64)
    v = yhat = y
    if case["post"] != "none":
        yhat, stats[:, 0], stats[:, 1] = _hat64(y, case["post"])
        v = yhat * (d["w_post"] + shift) + d.get("b_post", 0.0)
    g = torch.ones(1, 1, device=y.device, dtype=torch.float64)
    if case["gate"] != "none":
        g = d["gate"].reshape(T, 1) if case["gate"] == "token" else d["gate"].reshape(-1, H)
    raw = g
    if case["gate"] != "none" and case["sigmoid"]:
        g = torch.sigmoid(g)
    if not case["bwd"]:
        h = s["h"].double() + alpha * g * mask * v
        x = None
        if case["pre"] != "none":
            stored = h.to(s["dt"]).double()
            x, stats[:, 2], stats[:, 3] = _hat64(stored, case["pre"])
            x = x * (d["w_pre"] + shift) + d.get("b_pre", 0.0)
        return {"h_out": h, "x_out": x, "stats": stats}
    out = {}
    D = s["dh_out"].double()
    if case["pre"] != "none":
        xhat, _, rstd = _hat64(s["h_out"].double(), case["pre"])
        dx = s["dx_out"].double()
        out["dw_pre"] = (dx * xhat).sum(0)
        if case["pre"] == "layer":
            out["db_pre"] = dx.sum(0)
        D = D + _hat_back64(xhat, rstd, dx * (d["w_pre"] + shift), case["pre"])
    out["dh"] = D
    if case["gate"] != "none":
        slope = torch.sigmoid(raw) * torch.sigmoid(-raw) if case["sigmoid"] else torch.ones_like(raw)
        dg = alpha * mask * v * D
        if case["gate"] == "channel":
            dg = dg.sum(0, keepdim=True)
        if case["gate"] == "token":
            dg = dg.sum(1, keepdim=True)
        out["dgate"] = (dg * slope).reshape(d["gate"].shape)
    e = alpha * g * mask * D
    if case["post"] != "none":
        out["dw_post"] = (e * yhat).sum(0)
        if case["post"] == "layer":
            out["db_post"] = e.sum(0)
        _, _, rstd = _hat64(y, case["post"])
        e = _hat_back64(yhat, rstd, e * (d["w_post"] + shift), case["post"])
    out["dy"] = e
    return out


def _hat_back64(hat, rstd, d, kind):
    n = hat.shape[1]
    r = d - hat * ((d * hat).sum(1) / n)[:, None]
    if kind == "layer":
        r = r - (d.sum(1) / n)[:, None]
    return r * rstd[:, None]


def _exact_linear(case, s):
    x, w = s["x"].double(), s["w"].double()
    mask = _mask64((case["T"], case["N"]), case, s["rng"])
    act = case["act"]
    if case["bwd"]:
        dz = s["dout"].double() * mask
        if act != "none":
            z = s["pre"].double().requires_grad_(True)  # the activation's slope, differentiated
            with torch.enable_grad():
                a = _act64(z, act)
                slope, = torch.autograd.grad(a.sum(), z)
            dz = dz * slope
        return {"dx": torch.matmul(dz, w), "dw": torch.matmul(dz.t().contiguous(), x),
                "dbias": None if s["b"] is None else dz.sum(0)}
    z = torch.matmul(x, w.t())
    if s["b"] is not None:
        z = z + s["b"].double()
    y = _act64(z, act) * mask
    if s["res"] is not None:
        y = y + s["res"].double()
    return {"y": y, "pre": z if act != "none" else None}


def _act64(z, act):
    f = torch.nn.functional
    return {"none": lambda: z, "relu": lambda: f.relu(z), "silu": lambda: f.silu(z),
            "gelu": lambda: f.gelu(z), "gelu_tanh": lambda: f.gelu(z, approximate="tanh")}[act]()

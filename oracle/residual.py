"""Plain float64 definitions of the residual-stream operators, in NumPy.

dropout        Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
               SC 2011) at counter (element / 8, offset + site), key = seed, 16 bits an element
residual_norm  h' = h + alpha g drop(post(y)), x' = pre(h')
linear         y = residual + drop(act(x w^T + b))

Each with its gradient, written out from the formula.
"""
from __future__ import annotations

import math

import numpy as np

MASK32 = (1 << 32) - 1


def philox4x32(ctr, key):
    """ctr: four arrays (or ints) of 32-bit words, key: two words. Ten rounds; four words out."""
    c = [np.asarray(v, dtype=np.uint64) for v in ctr]
    k0, k1 = int(key[0]), int(key[1])
    lo, sh = np.uint64(MASK32), np.uint64(32)
    for _ in range(10):
        a = c[0] * np.uint64(0xD2511F53)
        b = c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k0), b & lo, (a >> sh) ^ c[3] ^ np.uint64(k1), a & lo]
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    return c


def dropout_threshold(p) -> int:
    """An element whose 16 bits are below this is dropped (p as the float32 the call takes)."""
    return int(math.floor(float(np.float32(p)) * 65536.0 + 0.5))


def dropout_keep(n, p, seed, offset, site=0):
    """[n] bool: which of the first n elements are kept."""
    ctr = np.arange((n + 7) // 8, dtype=np.uint64)
    off = (int(offset) + int(site)) & ((1 << 64) - 1)
    seed = int(seed) & ((1 << 64) - 1)
    words = philox4x32((ctr & np.uint64(MASK32), ctr >> np.uint64(32), off & MASK32, off >> 32),
                       (seed & MASK32, seed >> 32))
    u16 = np.empty((ctr.size, 8), dtype=np.uint64)
    for i, w in enumerate(words):
        u16[:, 2 * i], u16[:, 2 * i + 1] = w & np.uint64(0xFFFF), w >> np.uint64(16)
    return u16.reshape(-1)[:n] >= np.uint64(dropout_threshold(p))


def dropout(v, p, seed, offset, site=0):
    """v with dropped elements 0 and the others scaled by 1 / P(keep)."""
    t = dropout_threshold(p)
    if t == 0:
        return np.array(v, dtype=np.float64)
    keep = dropout_keep(v.size, p, seed, offset, site).reshape(v.shape)
    return np.where(keep, np.asarray(v, np.float64) * (65536.0 / (65536 - t)), 0.0)


# ---- norms: kind "rms" or "layer"; rows along the last axis
def norm_stats(u, kind, eps):
    mean = u.mean(-1) if kind == "layer" else np.zeros(u.shape[:-1])
    return mean, 1.0 / np.sqrt(((u - mean[..., None]) ** 2).mean(-1) + eps)


def norm(u, kind, eps, w, b=None):
    mean, rstd = norm_stats(u, kind, eps)
    v = (u - mean[:, None]) * rstd[:, None] * w
    return v if b is None else v + b


def norm_bwd(u, kind, eps, w, dv):
    """(du, dw, db) of norm() from the gradient dv at its output."""
    mean, rstd = norm_stats(u, kind, eps)
    hat = (u - mean[:, None]) * rstd[:, None]
    d = dv * w
    du = d - hat * (d * hat).mean(-1, keepdims=True)
    if kind == "layer":
        du = du - d.mean(-1, keepdims=True)
    return du * rstd[:, None], (dv * hat).sum(0), dv.sum(0)


def _gate(gate, kind, sigmoid):
    if kind == "none":
        return 1.0, 1.0
    raw = gate[:, None] if kind == "token" else gate
    if not sigmoid:
        return raw, np.ones_like(raw)
    g = 1.0 / (1.0 + np.exp(-raw))
    return g, g * (1.0 - g)


def residual_norm(h, y, prm, post="none", pre="rms", gate="none", gate_sigmoid=False, alpha=1.0,
                  eps=1e-5, weight_shift=0.0, drop=(0.0, 0, 0, 0)):
    """(h', v, g drop(v)): the stream after the block; pre(h') is norm() of h' as stored."""
    if y is None:
        return h, None, None
    v = y if post == "none" else norm(y, post, eps, weight_shift + prm["w_post"], prm.get("b_post"))
    g, _ = _gate(prm.get("gate"), gate, gate_sigmoid)
    add = g * dropout(v, *drop)
    return (0.0 if h is None else h) + alpha * add, v, add


def residual_norm_bwd(dh_out, dx_out, h_out, y, prm, post="none", pre="rms", gate="none",
                      gate_sigmoid=False, alpha=1.0, eps=1e-5, weight_shift=0.0,
                      drop=(0.0, 0, 0, 0)):
    """Gradients {dh, dy, dw_post, db_post, dgate, dw_pre, db_pre} (those that exist)."""
    out = {}
    D = 0.0 if dh_out is None else dh_out
    if pre != "none":
        du, dw, db = norm_bwd(h_out, pre, eps, weight_shift + prm["w_pre"], dx_out)
        D = D + du
        out["dw_pre"] = dw
        if pre == "layer":
            out["db_pre"] = db
    out["dh"] = D
    if y is None:
        return out
    v = y if post == "none" else norm(y, post, eps, weight_shift + prm["w_post"], prm.get("b_post"))
    g, slope = _gate(prm.get("gate"), gate, gate_sigmoid)
    if gate != "none":
        dg = alpha * dropout(v, *drop) * D
        if gate == "channel":
            dg = dg.sum(0)
        if gate == "token":
            dg = dg.sum(1, keepdims=True)
        out["dgate"] = (dg * slope).reshape(prm["gate"].shape)
    e = dropout(alpha * g * D, *drop)
    if post != "none":
        e, out["dw_post"], db = norm_bwd(y, post, eps, weight_shift + prm["w_post"], e)
        if post == "layer":
            out["db_post"] = db
    out["dy"] = e
    return out


# ---- linear
def act(z, kind):
    """(act(z), act'(z))"""
    from scipy.special import erf
    if kind == "none":
        return z, np.ones_like(z)
    if kind == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(z.dtype)
    if kind == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    if kind == "gelu":
        phi = 0.5 * (1.0 + erf(z * math.sqrt(0.5)))
        return z * phi, phi + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = np.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def linear(x, w, b=None, residual=None, kind="none", drop=(0.0, 0, 0, 0)):
    """(y, z) with z = x w^T + b, y = residual + drop(act(z))."""
    z = x @ w.T if b is None else x @ w.T + b
    y = dropout(act(z, kind)[0], *drop)
    return (y if residual is None else y + residual), z


def linear_bwd(dy, x, w, z, kind="none", drop=(0.0, 0, 0, 0)):
    """(dz, dx, dw, db)"""
    dz = dropout(dy, *drop)
    if kind != "none":
        dz = dz * act(z, kind)[1]
    return dz, dz @ w, dz.T @ x, dz.sum(0)

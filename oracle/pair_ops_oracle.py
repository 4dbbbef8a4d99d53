"""fp64 CPU definitions of the operators around the layer, and their derivatives.

Plain numpy, written from the definitions in include/trimul.h: the relative
position bias by buckets, the residual step with its two norms, and the norm
over many gradients with clipping.  The derivatives are the textbook ones of
each step, in fp64; test_oracle_pair_ops.py checks them against differences.
"""

from fractions import Fraction

import numpy as np


# ------------------------------------------------------------------ relative position bias
def log_bucket(n: int, K: int, M: int) -> int:
    """The one-sided LOG bucket of a distance n >= 0, decided in whole numbers."""
    E = K // 2
    if n < E:
        return n
    if n >= M:
        return K - 1
    k = 0  # the largest k with (n / E)^(K - E) >= (M / E)^k
    while k + 1 < K - E and Fraction(n, E) ** (K - E) >= Fraction(M, E) ** (k + 1):
        k += 1
    return E + k


def buckets(kind, M, num, two, q_pos, k_pos, q_group=None, k_group=None):
    """[B, I, J] table rows; -1 for padding.  num: the buckets without the one for different groups."""
    d = q_pos.astype(np.int64)[:, :, None] - k_pos.astype(np.int64)[:, None, :]
    if kind == "linear":
        b = np.clip(d, -M, M) + M if two else np.clip(d, 0, M)
    else:
        K = num // 2 if two else num
        lut = np.array([log_bucket(n, K, M) for n in range(M + 1)])
        b = lut[np.minimum(np.abs(d) if two else np.maximum(d, 0), M)]
        if two:
            b = b + K * (d < 0)
    if q_group is not None:
        gq, gk = q_group[:, :, None], k_group[:, None, :]
        b = np.where(gq != gk, num, b)
        b = np.where((gq < 0) | (gk < 0), -1, b)
    return b


def relpos_forward(table, b, base=None, layout="pair"):
    v = np.where((b >= 0)[..., None], table[np.maximum(b, 0)], 0.0)
    v = v if layout == "pair" else np.moveaxis(v, 3, 1)
    return v if base is None else v + base


def relpos_backward(dout, b, rows, layout="pair"):
    """(dtable, the sums of |dout| alike)."""
    d = dout if layout == "pair" else np.moveaxis(dout, 1, 3)
    out = np.zeros((2, rows, d.shape[-1]))
    on = b >= 0
    np.add.at(out[0], b[on], d[on])
    np.add.at(out[1], b[on], np.abs(d[on]))
    return out[0], out[1]


# ------------------------------------------------------------------ residual step
def _norm(v, kind, eps):
    if kind is None:
        return v, None
    c = v - v.mean(-1, keepdims=True) if kind == "layer" else v
    r = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    return c * r, r


def _norm_back(t, hat, r, kind):
    if kind is None:
        return t
    m1 = t.mean(-1, keepdims=True) if kind == "layer" else 0.0
    return r * (t - m1 - hat * (t * hat).mean(-1, keepdims=True))


def _parts(x, u, p, post, gate, sigmoid, mask, scale, eps):
    D = x.shape[-1]
    m = np.ones(x.shape[:3]) if mask is None else mask
    real = (m != 0)[..., None]
    u = np.where(real, u, 0.0)
    g = np.ones(D) if gate is None else 1 / (1 + np.exp(-gate)) if sigmoid else gate
    g = np.where(real, np.broadcast_to(g, x.shape), 0.0)
    hat, r = _norm(u, post, eps)
    y = hat * p.get("post_gamma", 1.0) + p.get("post_beta", 0.0)
    return m[..., None] * scale, real, g, hat, r, y, p.get("channel", np.ones(D))


def residual_forward(x, u, p, post=None, pre=None, gate=None, sigmoid=False, mask=None, scale=1.0, eps=1e-5):
    """(out, normed or None)."""
    k, real, g, _, _, y, ch = _parts(x, u, p, post, gate, sigmoid, mask, scale, eps)
    out = np.where(real, x + k * ch * g * y, x)
    if pre is None:
        return out, None
    hat, _ = _norm(np.where(real, out, 0.0), pre, eps)
    return out, np.where(real, hat * p.get("pre_gamma", 1.0) + p.get("pre_beta", 0.0), 0.0)


def residual_backward(x, u, dout, p, post=None, pre=None, gate=None, sigmoid=False, mask=None, scale=1.0, eps=1e-5,
                      dnormed=None):
    """dx, du, dgate (of every pair), and each parameter's gradient with the sum of its terms' magnitudes."""
    k, real, g, hat, r, y, ch = _parts(x, u, p, post, gate, sigmoid, mask, scale, eps)
    terms = {}
    d = dout.copy()
    if pre is not None:
        dn = np.where(real, dnormed, 0.0)
        xh, xr = _norm(np.where(real, x, 0.0) + k * ch * g * y, pre, eps)
        terms["pre_gamma"], terms["pre_beta"] = dn * xh, dn
        d = np.where(real, d + _norm_back(dn * p.get("pre_gamma", 1.0), xh, xr, pre), d)
    dx = d
    d = np.where(real, d, 0.0)
    kd = k * d
    terms["channel"] = kd * y * g
    dg = kd * y * ch * (g * (1 - g) if sigmoid else 1.0)
    dy = kd * ch * g
    terms["post_gamma"], terms["post_beta"] = dy * hat, dy
    du = _norm_back(dy * p.get("post_gamma", 1.0), hat, r, post)
    return dx, du, dg, {n: (t.sum((0, 1, 2)), np.abs(t).sum((0, 1, 2))) for n, t in terms.items()}


# ------------------------------------------------------------------ gradient norm and clipping
def grad_norm(tensors, inf=False):
    if inf:
        return max([np.abs(t).max() for t in tensors if t.size], default=0.0)
    return np.sqrt(sum((t.astype(np.longdouble) ** 2).sum() for t in tensors)) if tensors else 0.0


def grad_clip(tensors, max_norm, inf=False):
    n = grad_norm(tensors, inf)
    c = min(1.0, max_norm / (n + 1e-6)) if np.isfinite(n) else 1.0
    return n, [t * c for t in tensors]

"""The fp64 definitions of the operators around the layer: their derivatives
against central differences, and the buckets against closed forms."""

import numpy as np
import pytest

from oracle import pair_ops_oracle as O


def test_linear_buckets():
    q = np.array([[0, 5, -2**31, 2**31 - 1]])
    b = O.buckets("linear", 3, 7, True, q, q)
    assert b[0, 0].tolist() == [3, 0, 6, 0]
    assert b[0, 1].tolist() == [6, 3, 6, 0]
    assert b[0, 2].tolist() == [0, 0, 3, 0]
    assert O.buckets("linear", 3, 4, False, q, q)[0, 1].tolist() == [3, 0, 3, 0]


def test_log_buckets_on_their_borders():
    # 16 buckets up to 128: from 8 on the borders are 8 * 2^(k/2), exactly 16, 32, 64 at even k
    got = [O.log_bucket(n, 16, 128) for n in (7, 8, 11, 12, 15, 16, 22, 23, 31, 32, 63, 64, 127, 128, 10**6)]
    assert got == [7, 8, 8, 9, 9, 10, 10, 11, 11, 12, 13, 14, 15, 15, 15]


def test_groups_and_padding():
    pos, g = np.arange(4)[None], np.array([[0, 0, 1, -1]])
    b = O.buckets("linear", 2, 5, True, pos, pos, g, g)
    assert b[0].tolist() == [[2, 1, 5, -1], [3, 2, 5, -1], [5, 5, 2, -1], [-1, -1, -1, -1]]


@pytest.mark.parametrize("post,pre", [(None, None), ("layer", "rms"), ("rms", "layer")])
@pytest.mark.parametrize("gate,sigmoid", [(None, False), ("pair", True), ("row", False)])
def test_residual_gradients_against_differences(post, pre, gate, sigmoid):
    rng = np.random.default_rng(5)
    B, I, J, D = 2, 2, 3, 8
    v = {"x": rng.normal(size=(B, I, J, D)), "u": rng.normal(size=(B, I, J, D))}
    p = {"channel": 1 + 0.1 * rng.normal(size=D)}
    for name, kind in (("post", post), ("pre", pre)):
        if kind:
            p[name + "_gamma"] = 1 + 0.1 * rng.normal(size=D)
        if kind == "layer":
            p[name + "_beta"] = 0.1 * rng.normal(size=D)
    if gate:
        v["gate"] = rng.normal(size=(B, I if gate == "pair" else 1, J, D))
    mask = np.ones((B, I, J))
    mask[0, 1, 2] = 0
    mask[1, 0, 0] = 0.5
    dout = rng.normal(size=(B, I, J, D))
    dn = rng.normal(size=(B, I, J, D)) if pre else None

    def loss(v, p):
        out, n = O.residual_forward(v["x"], v["u"], p, post, pre, v.get("gate"), sigmoid, mask, 0.7)
        return (out * dout).sum() + (0.0 if n is None else (n * dn).sum())

    dx, du, dg, dp = O.residual_backward(v["x"], v["u"], dout, p, post, pre, v.get("gate"), sigmoid, mask, 0.7, 1e-5, dn)
    got = {"x": dx, "u": du, "gate": dg if gate == "pair" else dg.sum(1, keepdims=True)}
    h = 1e-5  # central differences: an error of h^2 and of 2^-52 / h, both near 1e-10 times the values
    for where, grads in ((v, {k: got[k] for k in v}), (p, {k: dp[k][0] for k in p})):
        for k, g in grads.items():
            e = rng.normal(size=where[k].shape)
            keep = where[k]
            where[k] = keep + h * e
            up = loss(v, p)
            where[k] = keep - h * e
            down = loss(v, p)
            where[k] = keep
            assert abs((up - down) / (2 * h) - (g * e).sum()) < 1e-7 * (1 + np.abs(g * e).sum()), k

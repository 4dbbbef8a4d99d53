"""The bounds of _residual.py see what they are there to see: mistakes planted in
the fp64 definitions of the residual step's gradients are outside them."""

import numpy as np
import pytest

from oracle import pair_ops_oracle as O
from tests import _residual as R

CASES = [(D, post, pre, gate) for D in (24, 136, 256) for post in ("layer", "rms") for pre in ("layer", "rms")
         for gate in (None, "sigmoid")]


def backward(D, post, pre, gate, rows=(1, 11, 13), seed=3):
    rng = np.random.default_rng(seed)
    shape = rows + (D,)
    x, u, dout, dn = (rng.normal(size=shape) for _ in range(4))
    p = {"channel": 0.5 + 0.2 * rng.normal(size=D)}
    for name, kind in (("post", post), ("pre", pre)):
        p[name + "_gamma"] = 1 + 0.2 * rng.normal(size=D)
        if kind == "layer":
            p[name + "_beta"] = 0.2 * rng.normal(size=D)
    g = None if gate is None else rng.normal(size=shape)
    dx, du, dg, dp = O.residual_backward(x, u, dout, p, post=post, pre=pre, gate=g, sigmoid=gate is not None, scale=0.75,
                                         dnormed=0.5 + dn)
    out = {"dx": (dx, None), "du": (du, None), **{k: dp[k] for k in p}}
    if g is not None:
        out["dgate"] = (dg, None)
    return out


def seen(ref, got, rows=143):
    return {k for k, (r, mag) in ref.items() if R.off(got[k][0], r, R.bound(k, r, mag, True, rows)) > 1.0}


def without_mean(t, hat, r, kind):
    return t if kind is None else r * (t - hat * (t * hat).mean(-1, keepdims=True))


def without_projection(t, hat, r, kind):
    return t if kind is None else r * (t - (t.mean(-1, keepdims=True) if kind == "layer" else 0.0))


def without_deviation(t, hat, r, kind):
    return O_norm_back(t, hat, r, kind) / (1.0 if kind is None else r) * (1.0 if kind is None else 1.01 * r)


O_norm_back = O._norm_back


def with_idle_lanes(D, gate):
    """The pre-norm's mean reaches the lanes past D, and from there the post-norm's."""
    idle = R.lanes(D) * 8 - D
    left = {}

    def back(t, hat, r, kind):
        if not left:
            left["d"] = -r * t.mean(-1, keepdims=True) * 0.75 * (1.0 if gate is None else 0.5)
            return O_norm_back(t, hat, r, kind)
        return r * (t - (t.sum(-1, keepdims=True) + idle * left["d"]) / D - hat * (t * hat).mean(-1, keepdims=True))

    return back


@pytest.mark.parametrize("D,post,pre,gate", CASES)
def test_planted_mistakes_are_seen(monkeypatch, D, post, pre, gate):
    ref = backward(D, post, pre, gate)
    assert not seen(ref, ref)
    for wrong in (without_mean, without_projection, without_deviation):
        if wrong is without_mean and "layer" not in (post, pre):
            continue
        with monkeypatch.context() as m:
            m.setattr(O, "_norm_back", wrong)
            assert seen(ref, backward(D, post, pre, gate)) & {"dx", "du"}, wrong.__name__
    if post == pre == "layer" and R.lanes(D) * 8 != D:
        with monkeypatch.context() as m:
            m.setattr(O, "_norm_back", with_idle_lanes(D, gate))
            assert "du" in seen(ref, backward(D, post, pre, gate))


@pytest.mark.parametrize("D,post,pre,gate", CASES)
def test_no_bound_accepts_zeros_or_another_scale(D, post, pre, gate):
    ref = backward(D, post, pre, gate)
    for k, (r, mag) in ref.items():
        limit = R.bound(k, r, mag, True, 143)
        assert limit <= R.SHARE * np.linalg.norm(r), k
        assert R.off(0.0 * r, r, limit) > 1.0 and R.off(1.1 * r, r, limit) > 1.0, k


def test_additions():
    assert R.additions(143, 24) == 1 + 64 + 1 + 5     # three blocks of 64 rows
    assert R.additions(304 * 8 * 7, 136) == 7 + 8 + 10 + 5

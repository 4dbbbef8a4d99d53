"""The residual step's gradients as whole tensors, against the fp64 definitions (bounds: _residual.py).

Widths that leave lanes of a row idle (all but the powers of two), with and
without a mask, over whole blocks of rows and a rest.
"""

import math

import numpy as np
import pytest
import torch

from oracle import pair_ops_oracle as O
from tests import _residual as R
from tests.test_gpu_pair_ops import RESIDUAL, f64, randn, residual_case, rng_of, spoil

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0**-24


@pytest.fixture(scope="module")
def P():
    from co_folding_pair_gb300 import pair_ops
    return pair_ops


def held(P, case, seed, second=False):
    _, x, u, p, kw, okw = residual_case(case, seed)
    g = rng_of(seed + 1)
    dout, dout2 = randn(g, *x.shape, dtype=case[4]), randn(g, *x.shape, dtype=case[4]) if second else None
    dn = 0.5 + randn(g, *x.shape) if case[6] else None  # its mean over the channels is not near 0
    dn = None if dn is None else dn.to(BF)
    spoil(kw["mask"], u, x, dn, kw["gate"])
    okw["gate"] = f64(kw["gate"])
    d = f64(dout) + (f64(dout2) if second else 0.0)
    dx, du, dg, rp = O.residual_backward(f64(x), f64(u), d, dnormed=f64(dn), **okw)
    got = P.trimul_residual_backward(x, u, dout, p, dnormed=dn, dout2=dout2, flags=P.FLAG_CHECK, **kw)
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    # padding pairs pass dout (+ dout2) on, whatever x holds there
    ref = {"dx": (dx, None), "du": (du, None), **{k: rp[k] for k in p}}
    if got["dgate"] is not None:
        ref["dgate"] = (dg, None)
    worst = {}
    for k, (r, mag) in ref.items():
        v = got[k] if mag is None else got["grads"][k]
        limit = R.bound(k, r, mag, v.dtype == BF, rows)
        assert limit <= R.SHARE * np.linalg.norm(r), f"{k}: the bound accepts anything"
        worst[k] = R.off(f64(v), r, limit)
    assert max(worst.values()) <= 1.0, {k: round(float(v), 3) for k, v in worst.items()}


# B, I, J, D, stream, post, pre, gate, sigmoid, channel, masked, affine: 143 rows are at least two blocks and a rest
IDLE = [(1, 11, 13, D, stream, "layer", "layer", gate, gate is not None, D == 96, False, True)
        for D in (24, 40, 96, 136, 200) for stream in (BF, F32) for gate in (None, "pair", "row")]


@pytest.mark.parametrize("case", IDLE, ids=lambda c: f"{c[3]}-{'fp32' if c[4] == F32 else 'bf16'}-{c[7]}")
def test_widths_with_idle_lanes(P, case):
    held(P, case, 51)


@pytest.mark.parametrize("post", [None, "layer", "rms"])
@pytest.mark.parametrize("pre", [None, "layer", "rms"])
@pytest.mark.parametrize("D", [16, 24, 56, 136, 256])
@pytest.mark.parametrize("masked", [False, True])
def test_every_pair_of_norms(P, post, pre, D, masked):
    for stream in (BF, F32):
        held(P, (2, 9, 17, D, stream, post, pre, "pair", masked, True, masked, True), 61, second=masked)


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("case", RESIDUAL, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}x{c[3]}-{c[5]}-{c[6]}-{c[7]}")
def test_the_cases_of_the_elementwise_test(P, case, second):
    if case[:3] == (1, 1, 1):
        case = (1, 1, 2) + case[3:]  # two pairs
    held(P, case, 22, second)


def test_pre_norm_parameters_against_differences(P):
    """normed is linear in pre_gamma and pre_beta, so a difference over any step is the derivative, but for rounding.

    A value of normed is rounded to bf16, by a number of root mean square at most 2^-8 / sqrt(3) of it; with values and
    weights near 1 the sum over n = 11520 of them is off by some 2^-8 / sqrt(3) 1.2 sqrt(n) = 0.29, the difference of
    two by 0.41, and over 2 h = 2 by 0.21: eight times that is 0.016 sqrt(n)."""
    g = rng_of(32)
    x, u = randn(g, 1, 10, 12, 96), randn(g, 1, 10, 12, 96, dtype=BF)
    for pre in ("layer", "rms"):
        p = {"post_gamma": 1 + 0.1 * randn(g, 96), "pre_gamma": 1 + 0.1 * randn(g, 96)}
        if pre == "layer":
            p["pre_beta"] = 0.1 * randn(g, 96)
        dn = randn(g, *x.shape, dtype=BF)
        kw = {"post_norm": "rms", "pre_norm": pre, "scale": 0.75}
        got = P.trimul_residual_backward(x, u, torch.zeros_like(x), p, dnormed=dn, **kw)["grads"]
        for k in ("pre_gamma", "pre_beta"):
            if k not in p:
                continue
            e = randn(g, 96)
            up, down = (float((P.trimul_residual_forward(x, u, {**p, k: p[k] + h * e}, **kw)[1].double() * dn.double()).sum())
                        for h in (1.0, -1.0))
            assert abs((up - down) / 2 - float((got[k].double() * e).sum())) < 0.016 * math.sqrt(x.numel()), (pre, k)


@pytest.mark.parametrize("sign", [1, -1])
def test_sigmoid_gates_of_large_logits(P, sign):
    """The gate alone (x = 0, u = 1): exp(-|x|) is off by at most 2 + 1.173 |x| ulp (the fast exponential's documented
    bound), the sum, reciprocal and product by 3 more; an ulp is at most 2^-23 of a value.  Results below the smallest
    normal number are 0.  1 - small has fp32's precision whatever small's."""
    logits = (sign * torch.linspace(0.0, 100.0, 2048, device="cuda")).to(BF).view(1, 16, 16, 8)
    x, u = torch.zeros(1, 16, 16, 8, device="cuda"), torch.ones(1, 16, 16, 8, dtype=BF, device="cuda")
    t = f64(logits)
    e = np.exp(-np.abs(t))
    small = e / (1 + e)
    ref = small if sign < 0 else 1 - small
    steps = 5 + 1.173 * np.abs(t)
    out = f64(P.trimul_residual_forward(x, u, gate=logits, gate_sigmoid=True)[0])
    assert (np.abs(out - ref) <= steps * 2.0**-23 * small + U * ref + 2.0**-126).all()
    # dgate = u small (1 - small), whichever the sign, rounded to bf16
    got = f64(P.trimul_residual_backward(x, u, torch.ones_like(x), gate=logits, gate_sigmoid=True)["dgate"])
    slope = small * (1 - small)
    assert (np.abs(got - slope) <= (2.0**-8 + (steps + 2) * 2.0**-23) * slope + 2.0**-126).all()

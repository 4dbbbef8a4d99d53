"""The residual step's gradients as whole tensors, against the fp64 definitions (bounds: _residual.py).

Widths that leave lanes of a row idle (all but the powers of two), with and
without a mask, over whole blocks of rows and a rest.
"""

import numpy as np
import pytest
import torch

from oracle import pair_ops_oracle as O
from tests import _residual as R
from tests.test_gpu_pair_ops import f64, randn, residual_case, rng_of, spoil

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


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

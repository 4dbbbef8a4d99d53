"""AdamW's 8-bit states bit for bit, and where gradients are not finite, on a GB300."""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16
# tensors of a few blocks, and what makes a thread block take one block of states a warp, two, or two with the next on their way
SIZES = {"one block": [1000, 300, 384], "two blocks": [700001, 1000, 384], "two ahead": [5400001, 1000, 384]}


@pytest.fixture(scope="module")
def P():
    from co_folding_pair_gb300 import train_ops
    return train_ops


def randn(g, n):
    return torch.randn(n, generator=g, device="cuda")


def decoded(opt, key):
    return (opt.state[key].float().view(-1, 128) * opt.state[key + "_scale"][:, None])


def bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t.view(torch.int32 if t.dtype == F32 else torch.int16 if t.dtype == BF else t.dtype)


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("form", list(SIZES))
def test_a_gradient_that_is_not_finite_stays_in_its_block(P, form, bad, rounding):
    """Without a norm: the block of states is not finite from then on, all of it, its parameters from the next step on;
    all other blocks are as without it, bit for bit."""
    sizes = SIZES[form]

    def run(at):
        g = torch.Generator(device="cuda")
        g.manual_seed(17)
        params, grads = [randn(g, n) for n in sizes], [0.01 * randn(g, n) for n in sizes]
        opt = P.AdamW(params, lr=1e-2, states="8bit", rounding=rounding, seed=5)
        opt.step(grads)
        good = [v.clone() for v in grads]
        for k, i in at:
            grads[k][i] = bad
        opt.step(grads)
        first = {k: v.clone() for k, v in opt.state.items()}, [p.clone() for p in params]
        if at:
            assert_blocks(opt, at)
        opt.step(good)
        if at:
            assert_blocks(opt, at)
        opt.step(good)
        return opt, params, first

    def block(opt, k, i):
        return opt.starts[k] // 128 + i // 128

    def assert_blocks(opt, at):
        for k, i in at:
            for key in "mv":
                n = min(128, sizes[k] - i // 128 * 128)  # (nothing stands behind a tensor's end)
                assert not torch.isfinite(decoded(opt, key)[block(opt, k, i), :n]).any(), (key, k, i)

    at = [(0, 130), (0, sizes[0] - 1), (1, 5), (2, 383)]
    opt, params, (s1, p1) = run(at)
    ref, want, (t1, q1) = run([])
    assert_blocks(opt, at)
    rows = torch.ones(opt.state["m"].numel() // 128, dtype=torch.bool, device="cuda")
    for k, i in at:
        rows[block(opt, k, i)] = False
    for state, other in ((s1, t1), (opt.state, ref.state)):
        for key in "mv":
            assert torch.equal(bits(state[key]).view(-1, 128)[rows], bits(other[key]).view(-1, 128)[rows])
            assert torch.equal(bits(state[key + "_scale"])[rows], bits(other[key + "_scale"])[rows])
    for k in range(3):
        bad_at = torch.zeros(sizes[k], dtype=torch.bool, device="cuda")
        for j, i in at:
            if j == k:
                bad_at[i] = True
        # in the step itself the others of the block move as they would
        assert torch.equal(bits(p1[k])[~bad_at], bits(q1[k])[~bad_at]) and not torch.isfinite(p1[k][bad_at]).any()
        for j, i in at:
            if j == k:
                bad_at[i // 128 * 128:i // 128 * 128 + 128] = True
        assert torch.equal(bits(params[k])[~bad_at], bits(want[k])[~bad_at]) and torch.isnan(params[k][bad_at]).all()

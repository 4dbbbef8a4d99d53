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


# ------------------------------------------------------------------ bit for bit
f = np.float32
B1, B2 = 0.9, 0.999


def moments(g, m, v, clip):
    """The new m and v, each operation rounded to fp32."""
    ge = g * f(clip)
    return f(B1) * m + f(1 - B1) * ge, f(B2) * v + (f(1 - B2) * ge) * ge


def e4m3_bytes(q):
    return torch.from_numpy(np.ascontiguousarray(q)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def packed(x, random16, roots):
    """The codes and scales of x, each operation rounded to fp32; random16: what decides between two neighbours, or None."""
    blocks = np.pad(x, (0, -len(x) % 128)).reshape(-1, 128)
    scale = np.maximum(np.abs(blocks).max(1), f(2.0**-90)) * (f(1) / f(448))
    q = x * np.repeat(f(1) / scale, 128)[: len(x)]
    if random16 is not None:
        a = np.abs(q)
        base = np.where(a < f(2.0**-6), f(2.0**-6), f(0))
        up = ((a + base).view(np.uint32) + (random16.astype(np.uint32) << np.uint32(4))) & np.uint32(0xFFF00000)
        q = np.copysign(up.view(f) - base, q)
    q = np.clip(q, f(-448), f(448))
    if roots:
        q = torch.from_numpy(np.ascontiguousarray(q)).to(torch.float8_e4m3fn).float().numpy()
        q = np.where(x > 0, np.maximum(q, f(2.0**-9)), q)
    return e4m3_bytes(q), scale


@pytest.mark.parametrize("n", [5, 1000, 131072, 700001, 5300003])
@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("wide", [False, True])
def test_states_are_those_of_plain_arithmetic(P, n, rounding, wide):
    """Codes and scales of two steps, and 32-bit states: the bits of fp32 arithmetic, operation by operation.  `wide`: numbers of
    all sizes in a block, their squares below and above fp32's normal range."""
    from oracle import train_ops_oracle as O
    r = np.random.default_rng(n)
    g = r.standard_normal(n).astype(f)
    if wide:
        g = (g * 10.0 ** r.uniform(-24, 18, n)).astype(f)
        g[:: 7] *= f(1e-3)
    opts = {}
    for states in ("8bit", "float32"):
        opts[states] = P.AdamW([torch.zeros(n, device="cuda")], states=states, rounding=rounding, seed=77, weight_decay=0.0, betas=(B1, B2))
    m = v = m32 = v32 = np.zeros(n, f)
    for t in (1, 2):
        ge = g if t == 1 else np.roll(g, 1)
        norm, most = f(3.0), 0.75 if t == 2 else None  # the second step clips
        clip = f(1) if t == 1 else f(most) * (f(1) / (norm + f(1e-6)))
        for opt in opts.values():
            opt.step([torch.from_numpy(ge.copy()).cuda()], norm=None if t == 1 else torch.full((), 3.0, device="cuda"), max_norm=most)
        with np.errstate(all="ignore"):
            m32, v32 = moments(ge, m32, v32, clip)
            m, v = moments(ge, m, v, clip)
            root = np.sqrt(v)
            h = O.random_bits(77, t, 0, np.arange(n)) if rounding == "stochastic" else None
            for key, x, b in (("m", m, None if h is None else h & np.uint64(0xFFFF)), ("v", root, None if h is None else h >> np.uint64(16))):
                codes, scale = packed(x, b, key == "v")
                state = opts["8bit"].state
                assert np.array_equal(state[key].view(torch.uint8)[:n].cpu().numpy(), codes), (key, t)
                assert np.array_equal(state[key + "_scale"].cpu().numpy(), scale), (key, t)
                held = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy() * np.repeat(scale, 128)[:n]
                m, v = (held, v) if key == "m" else (m, held * held)
        assert np.array_equal(opts["float32"].state["m"][:n].cpu().numpy(), m32) and np.array_equal(opts["float32"].state["v"][:n].cpu().numpy(), v32)


def test_roots_of_many_numbers(P):
    """A block's largest root is in its scale with all its bits: a million of them, of all sizes whose squares are normal numbers."""
    blocks = 1 << 20
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    top = torch.rand(blocks, generator=g, device="cuda") + 1.0
    top = top * torch.exp2(torch.randint(-58, 60, (blocks,), generator=g, device="cuda").float())
    grad = (top[:, None] * torch.linspace(0.1, 1.0, 128, device="cuda")).contiguous().view(-1)  # (linspace ends at 1: `top` is among them)
    opt = P.AdamW([torch.zeros(blocks * 128, device="cuda")], states="8bit", rounding="nearest", betas=(B1, B2))
    opt.step([grad])
    big = grad.view(-1, 128).amax(1).cpu().numpy()
    v = (f(1 - B2) * big) * big
    assert np.array_equal(opt.state["v_scale"].cpu().numpy(), np.sqrt(v) * (f(1) / f(448)))

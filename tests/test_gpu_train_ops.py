"""AdamW against its fp64 definition, on a GB300.

Tolerances, U = 2^-24: m is two products and a sum of numbers that are off by at most 4 U (the factors 1 - b
rounded, the clipping factor a quotient, the gradient's product with it): 8 U of |b1 m| + |(1 - b1) g|.  v has one product
more: 12 U of itself (all its terms are positive).  The step divides m by a root (approximate, 2 ulp = 4 U, of v's 12 U / 2 and of
the correction's) and multiplies by lr / (1 - b1^t): each correction is off by 2 U of its exponent, whose
effect on 1 - b^t is no more than that, 2 U of expm1f and U of the quotient; eps, the sum, the quotient (2 ulp) and the product add 8 U:
40 U of lr / (1 - b1^t) (|b1 m| + |(1 - b1) g|) / denominator.  p's own product and sums: 6 U |p|.  Then each output is
rounded once: eps / 2 of its type.

A code of an 8-bit state is the rounding of y = x / scale, which is off by 16 U of x's magnitudes over the scale (x
above, the scale's quotient and reciprocal 4 U): it has to lie between the roundings, with the same random
bits, of y less that and y plus that.
"""

import math

import numpy as np
import pytest
import torch

from oracle import train_ops_oracle as O

pytestmark = pytest.mark.gpu
BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16
U = 2.0**-24
HALF = {BF: 2.0**-8, F32: 2.0**-24, F16: 2.0**-11}
TINY = {BF: 0.0, F32: 0.0, F16: 2.0**-25}  # half of fp16's least number


@pytest.fixture(scope="module")
def P():
    from co_folding_pair_gb300 import train_ops
    return train_ops


@pytest.fixture(scope="module")
def R():
    from co_folding_pair_gb300 import pair_ops
    return pair_ops


def rng_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def within(got, ref, tol, what):
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / (tol + 1e-300)):.3g} of the bound"


# ------------------------------------------------------------------ AdamW
HYPER = {"lr": 3e-3, "betas": (0.9, 0.999), "eps": 1e-8}


def make(P, g, sizes, pdt=F32, gdt=F32, cdt=None, offset=0, states="float32", rounding="stochastic", count=0, decay=0.01, seed=7, **kw):
    """An AdamW over tensors of `sizes` that begin `offset` elements past the allocator's boundary, and gradients."""
    def views(dt, scale):
        return [(scale * randn(g, n + offset)).to(dt)[offset:] for n in sizes]

    params, grads = views(pdt, 0.1), [v * (10.0 ** (k % 5 - 3)) for k, v in enumerate(views(gdt, 1.0))]
    if offset:
        grads = [torch.cat([v.new_zeros(offset), v])[offset:] for v in grads]
    copies = None if cdt is None else [None if k % 3 == 2 else torch.zeros(n + offset, dtype=cdt, device="cuda")[offset:] for k, n in enumerate(sizes)]
    opt = P.AdamW(params, weight_decay=[decay * (k % 2) for k in range(len(sizes))], states=states, copies=copies, rounding=rounding,
                  seed=seed, **{**HYPER, **kw})
    opt.state["count"].fill_(count)
    if count:
        for n, a, v in zip(sizes, opt.starts, grads):
            m, r = 0.5 * v.float() * randn(g, n), v.float().abs() * torch.exp(randn(g, n))
            if states == "float32":
                opt.state["m"][a:a + n], opt.state["v"][a:a + n] = m, r * r
            else:
                for key, x in (("m", m), ("v", r)):
                    s = torch.nn.functional.pad(x, (0, -n % 128)).view(-1, 128).abs().amax(1).clamp(min=2.0**-90) / 448
                    opt.state[key + "_scale"][a // 128:a // 128 + len(s)] = s
                    opt.state[key][a:a + n] = (x / s.repeat_interleave(128)[:n]).to(torch.float8_e4m3fn)
    return opt, params, grads, copies


def snapshot(opt, params, sizes):
    state = {k: f64(v.float() if v.dtype == torch.float8_e4m3fn else v) for k, v in opt.state.items()}
    return [f64(p) for p in params], state


def held(state, key, a, n, eight):
    """What a state stands for."""
    x = state[key][a:a + n]
    return O.dequantized(x, state[key + "_scale"][a // 128:a // 128 + -(-n // 128)]) if eight else x


def check_step(opt, before, params, grads, copies, sizes, t, seed=7, norm=None, max_norm=None, lr=None, decay=0.01):
    p0, s0 = before
    _, s1 = snapshot(opt, params, sizes)
    eight, stochastic = opt.eight, opt._p.rounding == 1
    clip = O.clip_factor(norm, max_norm)
    assert s1["count"] == t
    for k, (n, a) in enumerate(zip(sizes, opt.starts)):
        m0, v0 = held(s0, "m", a, n, eight), held(s0, "v", a, n, eight)
        v0 = v0 * v0 if eight else v0
        p, m, v, mag, move = O.adamw(p0[k], f64(grads[k]), m0, v0, t, lr or HYPER["lr"], HYPER["betas"], HYPER["eps"], decay * (k % 2), clip)
        tol = 6 * U * np.abs(p0[k]) + 40 * U * move
        dt = params[k].dtype
        bits = O.random_bits(seed, t, k, np.arange(n))
        if dt == BF and stochastic:
            lo, hi = (O.bf16_at_random(p + d, O.pcg(bits) & np.uint64(0xFFFF)) for d in (-tol, tol))
            got = f64(params[k])
            assert ((got >= lo) & (got <= hi)).all(), k
        else:
            within(params[k], p, HALF[dt] * (np.abs(p) + tol) + tol, f"params[{k}]")
        if copies is not None and copies[k] is not None:
            dt = copies[k].dtype
            within(copies[k], p, HALF[dt] * (np.abs(p) + tol) + tol + TINY[dt], f"copies[{k}]")
        if not eight:
            within(opt.state["m"][a:a + n], m, 8 * U * mag, f"m[{k}]")
            within(opt.state["v"][a:a + n], v, 12 * U * v, f"v[{k}]")
            continue
        for key, x, err, b in (("m", m, 8 * U * mag, bits & np.uint64(0xFFFF)), ("v", np.sqrt(v), 12 * U * np.sqrt(v), bits >> np.uint64(16))):
            scale = O.scales(x)
            got = s1[key + "_scale"][a // 128:a // 128 + len(scale)]
            assert (np.abs(got - scale) <= O.blocks(err).max(1) / 448 + 4 * U * scale).all(), (k, key)
            full = np.repeat(scale, 128)[:n]
            y, off = x / full, (err + 8 * U * np.abs(x)) / full + np.repeat(O.blocks(err).max(1) / 448 / scale, 128)[:n] * np.abs(x) / full
            rounded = (lambda q: O.e4m3_at_random(q, b / 65536.0)) if stochastic else O.e4m3
            lo, hi = rounded(y - off), rounded(y + off)
            if key == "v":
                lo, hi = (np.where(v > 0, np.maximum(q, 2.0**-9), q) for q in (lo, hi))
            q = s1[key][a:a + n]
            assert ((q >= lo) & (q <= hi)).all(), (k, key, np.flatnonzero((q < lo) | (q > hi))[:5])


SIZES = [1, 0, 127, 128, 129, 1023, 1024, 1025, 4099, 70000]


@pytest.mark.parametrize("states", ["float32", "8bit"])
@pytest.mark.parametrize("pdt,gdt,cdt,offset,rounding,count", [
    (F32, F32, None, 0, "nearest", 0),
    (F32, F32, BF, 0, "stochastic", 1000),
    (F32, BF, F16, 0, "stochastic", 0),
    (F32, F16, BF, 1, "nearest", 12),
    (BF, BF, None, 0, "stochastic", 300),
    (BF, F32, None, 3, "stochastic", 0),
    (BF, F16, None, 0, "nearest", 70000),
], ids=str)
def test_adamw(P, states, pdt, gdt, cdt, offset, rounding, count):
    opt, params, grads, copies = make(P, rng_of(3), SIZES, pdt, gdt, cdt, offset, states, rounding, count)
    for t in (count + 1, count + 2):
        before = snapshot(opt, params, SIZES)
        opt.step(grads, flags=P.FLAG_CHECK)
        check_step(opt, before, params, grads, copies, SIZES, t)


@pytest.mark.parametrize("pdt,gdt,cdt,offset,rounding", [(F32, F32, BF, 0, "stochastic"), (BF, BF, None, 0, "nearest"), (F32, F16, None, 1, "stochastic")], ids=str)
def test_adamw_8bit_where_blocks_take_more_than_one_turn(P, pdt, gdt, cdt, offset, rounding):
    """Warps with two blocks of states each, one, a part of one, and none."""
    sizes = [600001, 130, 127, 128, 129, 256, 257, 383, 384, 385, 1, 2047, 2048, 2049, 0, 4095]
    opt, params, grads, copies = make(P, rng_of(31), sizes, pdt, gdt, cdt, offset, "8bit", rounding, 3)
    for t in (4, 5):
        before = snapshot(opt, params, sizes)
        opt.step(grads, flags=P.FLAG_CHECK)
        check_step(opt, before, params, grads, copies, sizes, t)


@pytest.mark.parametrize("pdt,gdt,cdt,offset", [(F32, F32, BF, 0), (BF, F32, None, 1)], ids=str)
@pytest.mark.parametrize("many", [False, True])
def test_adamw_8bit_where_blocks_take_many_turns(P, pdt, gdt, cdt, offset, many):
    """Past five million numbers, from tensor to tensor within a block's turns; with more tensors than the small table has."""
    sizes = [70001 + 128 * k for k in range(70)] + [1, 0, 136, 2047, 2049] if many else [3000001, 2049, 128, 2100000, 1, 0, 257]
    opt, params, grads, copies = make(P, rng_of(32), sizes, pdt, gdt, cdt, offset, "8bit", "stochastic", 3)
    for t in (4, 5):
        before = snapshot(opt, params, sizes)
        opt.step(grads, flags=P.FLAG_CHECK)
        check_step(opt, before, params, grads, copies, sizes, t)


@pytest.mark.parametrize("states", ["float32", "8bit"])
@pytest.mark.parametrize("n", [64, 65, 384, 385, 900])
def test_adamw_many_tensors(P, states, n):
    """One launch's table and more than that; the step is counted once."""
    sizes = [(37 * k) % 700 for k in range(n)]
    opt, params, grads, copies = make(P, rng_of(n), sizes, cdt=BF, states=states, count=5)
    before = snapshot(opt, params, sizes)
    opt.step(grads)
    check_step(opt, before, params, grads, copies, sizes, 6)


@pytest.mark.parametrize("states", ["float32", "8bit"])
@pytest.mark.parametrize("share", [0.3, 5.0])
def test_adamw_clips_in_its_own_pass(P, R, states, share):
    """Against the definition with the clipping factor, and (32 bits, in place) against clip and then a step."""
    opt, params, grads, copies = make(P, rng_of(11), SIZES, states=states, count=40)
    gs = R.GradSet(grads)
    norm = gs.norm()
    most = share * float(norm)
    before, p0 = snapshot(opt, params, SIZES), [p.clone() for p in params]
    opt.step(gs, norm=norm, max_norm=most)
    check_step(opt, before, params, grads, copies, SIZES, 41, norm=float(norm), max_norm=most)
    gs.clip(most)
    for p, q in zip(params, p0):
        p.data, q.data = q.data, p.data  # q: after the step
    other = P.AdamW(params, weight_decay=[0.01 * (k % 2) for k in range(len(SIZES))], states=states, seed=7, **HYPER)
    for k, v in other.state.items():
        v.copy_(torch.from_numpy(np.asarray(before[1][k])).to(v.dtype))
    other.step(gs)
    for p, q in zip(params, p0):
        within(p, f64(q), 2e-4 * HYPER["lr"] + 12 * U * np.abs(f64(q)), "two passes")  # 40 U of steps below 80 lr


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_adamw_leaves_all_as_it_is_where_the_norm_is_not_finite(P, R, bad):
    opt, params, grads, copies = make(P, rng_of(12), SIZES, cdt=BF, states="8bit", count=4)
    grads[-1][5] = bad
    gs = R.GradSet(grads)
    before = [t.clone() for t in params + [c for c in copies if c is not None]] + [v.view(torch.uint8 if v.dtype == torch.float8_e4m3fn else v.dtype).clone() for v in opt.state.values()]
    opt.step(gs, norm=gs.norm(), max_norm=1.0)
    after = params + [c for c in copies if c is not None] + [v.view(torch.uint8 if v.dtype == torch.float8_e4m3fn else v.dtype) for v in opt.state.values()]
    assert all(torch.equal(a, b) for a, b in zip(before, after)) and int(opt.state["count"]) == 4
    grads[-1][5] = 1.0
    opt.step(gs, norm=gs.norm(), max_norm=1.0)
    assert int(opt.state["count"]) == 5


def test_adamw_8bit_states_at_their_ends(P):
    """Gradients of zero, a block with one large value among small ones, subnormals, and a long run of steps."""
    n = 512
    g = torch.zeros(n, device="cuda")
    g[128] = 100.0
    g[129:256] = 1e-7
    g[256:384] = 1e-40
    g[384:512] = 1e18
    p = torch.zeros(n, device="cuda")
    opt = P.AdamW([p], lr=1e-3, weight_decay=0.0, states="8bit", seed=3)
    for _ in range(50):
        opt.step([g])
    assert torch.isfinite(p).all() and (p[:128] == 0).all()
    # no step is more than lr / (1 - b1) by AdamW's own bound for constant gradients (they are lr each), codes off by an eighth or kept above zero
    assert float(p.abs().max()) <= 50 * 1e-3 * 1.3
    v = opt.state["v"].float()
    assert (v[:128] == 0).all() and (v[128:256] > 0).all() and (v[384:] == 448).all()


@pytest.mark.parametrize("states", ["float32", "8bit"])
def test_adamw_of_tiny_gradients(P, states):
    """Squares below fp32's normal range, with an eps smaller than their roots: the step is still lr's size."""
    g = torch.tensor([1e-18, -3e-19, 2e-17, 1e-15], device="cuda").repeat(64)
    p = torch.zeros(256, device="cuda")
    opt = P.AdamW([p], lr=1.0, weight_decay=0.0, states=states, betas=(0.9, 0.999), eps=1e-30, rounding="nearest")
    opt.step([g])
    g64 = f64(g)
    v = (g64 * g64 * 1e-3).astype(np.float32).astype(np.float64)  # subnormal: in steps of 2^-149
    want = -(0.1 * g64 / 0.1) / (np.sqrt(v / 1e-3) + 1e-30)
    # a subnormal v is off by 2 steps of 2^-149, its root by half that share
    within(p, want, (2.0**-149 / v + 64 * U) * np.abs(want), "p")


def test_adamw_random_rounding_is_fair(P):
    """The mean over many elements is the value: a code's place is uniform, so its variance is at most step^2 / 4 and
    the mean of n is within 5 step / (2 sqrt n) (5 deviations), the bits' grid adding step 2^-16."""
    n = 1 << 20
    g = torch.full((n,), 0.37, device="cuda")
    g[::128] = 1.0  # each block's scale
    p = torch.full((n,), 1.0 + 1.0 / 512, device="cuda").to(BF)
    p.fill_(1.0)
    opt = P.AdamW([p], lr=1e-3, weight_decay=0.0, states="8bit", seed=99)
    opt.step([g])
    m = opt.state["m"].float().view(-1, 128)[:, 1:] * opt.state["m_scale"][:, None]
    r = opt.state["v"].float().view(-1, 128)[:, 1:] * opt.state["v_scale"][:, None]
    for x, want, top in ((m, 0.1 * 0.37, 0.1), (r, math.sqrt(1e-3) * 0.37, math.sqrt(1e-3))):
        step = 16 * top / 448  # e4m3 in [128, 256): 0.37 * 448 = 166
        values = torch.unique((x / (top / 448)).round())
        assert values.tolist() == [160.0, 176.0]
        assert abs(float(x.double().mean()) - want) <= 5 * step / (2 * math.sqrt(x.numel())) + step * 2.0**-16 + 16 * U * want
    q = p.double()  # 1 - 1e-3 lies between 1 - 2^-8 and 1 (steps of 2^-8 below 1)
    assert sorted(torch.unique(q).tolist()) == [1 - 2.0**-8, 1.0]
    assert abs(float(q.mean()) - 0.999) <= 5 * 2.0**-8 / (2 * math.sqrt(n)) + 2.0**-24


def test_adamw_seeds_and_repeats(P):
    def after(seed, steps=2):
        opt, params, grads, _ = make(P, rng_of(5), [5000, 300], pdt=BF, states="8bit", seed=seed)
        for _ in range(steps):
            opt.step(grads)
        return torch.cat([p.float() for p in params] + [opt.state["m"].float(), opt.state["v"].float()])
    assert torch.equal(after(1), after(1))
    assert not torch.equal(after(1), after(2))


@pytest.mark.parametrize("states", ["float32", "8bit"])
def test_adamw_in_a_graph(P, R, states):
    """Captured with its norm and a learning rate on the device: replays are the steps that eager calls take."""
    def setup():
        opt, params, grads, copies = make(P, rng_of(21), SIZES, cdt=BF, states=states, count=3)
        return opt, params, grads, torch.full((), 1e-3, device="cuda"), R.GradSet(grads)

    a, pa, ga, la, sa = setup()
    b, pb, gb, lb, sb = setup()
    norm = torch.zeros((), device="cuda")
    sa.norm(norm=norm)
    a.step(sa, lr=la, norm=norm, max_norm=0.5)
    sb.norm(norm=norm)
    b.step(sb, lr=lb, norm=norm, max_norm=0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.norm(norm=norm)
        a.step(sa, lr=la, norm=norm, max_norm=0.5)
    for k in range(3):
        for x, y in zip(ga, gb):
            fresh = randn(rng_of(100 + k), *x.shape)
            x.copy_(fresh)
            y.copy_(fresh)
        la.fill_(1e-3 * (k + 1))
        lb.fill_(1e-3 * (k + 1))
        graph.replay()
        n2 = sb.norm()
        b.step(sb, lr=lb, norm=n2, max_norm=0.5)
    assert int(a.state["count"]) == int(b.state["count"]) == 7
    assert all(torch.equal(x, y) for x, y in zip(pa, pb))
    assert all(torch.equal(a.state[k].float(), b.state[k].float()) for k in a.state)


def test_adamw_on_another_stream(P):
    """After work on that stream that is still running when the call is made."""
    opt, params, grads, copies = make(P, rng_of(22), SIZES, states="8bit", count=2)
    before = snapshot(opt, params, SIZES)
    s, late = torch.cuda.Stream(), [torch.zeros_like(v) for v in grads]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        for x, y in zip(late, grads):
            x.copy_(y)
    opt.step(late, stream=s)
    s.synchronize()
    check_step(opt, before, params, grads, copies, SIZES, 3)


@pytest.mark.parametrize("states", ["float32", "8bit"])
def test_adamw_writes_nothing_else(P, states):
    """Parameters and copies as parts of larger buffers, and the states of neighbouring tensors."""
    sizes = [1, 5, 130, 1031]
    opt, params, grads, _ = make(P, rng_of(31), sizes, states=states, count=2)
    bufs, views = [], []
    for k, n in enumerate(sizes):
        for dt in (F32, BF):
            buf = torch.full((n + 64,), 7.25, dtype=dt, device="cuda")
            bufs.append(buf)
            views.append(buf[32 + k:32 + k + n])
    opt = P.AdamW(views[::2], copies=views[1::2], states=states, **HYPER)
    for v in opt.state.values():
        v.fill_(2.0 if v.dtype != torch.int32 else 0)
    opt.step(grads)
    for k, n in enumerate(sizes):
        for buf in bufs[2 * k:2 * k + 2]:
            assert (buf[:32 + k] == 7.25).all() and (buf[32 + k + n:] == 7.25).all()
        a, end = opt.starts[k], opt.starts[k] + -(-n // 128) * 128
        for key in "mv":
            assert (opt.state[key][a + n:end].float() == 2.0).all()
            assert not (opt.state[key][a:a + n].float() == 2.0).all()


def test_adamw_past_32_bits(P):
    """A tensor of more than 2^32 elements: its last ones against the definition."""
    n = (1 << 32) + 1000
    g = torch.zeros(n, dtype=BF, device="cuda")
    p = torch.ones(n, dtype=BF, device="cuda")
    g[-2000:] = randn(rng_of(8), 2000, dtype=BF)
    opt = P.AdamW([p], states="8bit", seed=7, weight_decay=0.01, **HYPER)
    opt.step([g])
    i = np.arange(n - 2000, n)
    bits = O.random_bits(7, 1, 0, i)
    z = np.zeros(2000)
    q, m, v, mag, move = O.adamw(z + 1, f64(g[-2000:]), z, z, 1, HYPER["lr"], HYPER["betas"], HYPER["eps"], 0.01)
    tol = 6 * U + 40 * U * move
    lo, hi = (O.bf16_at_random(q + d, O.pcg(bits) & np.uint64(0xFFFF)) for d in (-tol, tol))
    got = f64(p[-2000:])
    assert ((got >= lo) & (got <= hi)).all()
    assert (opt.state["m"][: n - 2000].view(torch.uint8) == 0).all()
    del g, p, opt
    torch.cuda.empty_cache()


def test_adamw_refusals(P, R):
    x, y = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    opt = P.AdamW([x])
    with pytest.raises(ValueError, match="2 grads for 1 params"):
        opt.step([y, y])
    with pytest.raises(Exception, match="its gradient has 8 elements, not 64"):
        opt.step([y[:8]])
    with pytest.raises(ValueError, match="both norm and max_norm"):
        opt.step([y], norm=torch.ones((), device="cuda"))
    with pytest.raises(ValueError, match="norm must be one float32"):
        opt.step([y], norm=torch.ones(()), max_norm=1.0)
    with pytest.raises(Exception, match="max_norm must be"):
        opt.step([y], norm=torch.ones((), device="cuda"), max_norm=-1.0)
    with pytest.raises(Exception, match="param overlaps grad"):
        opt.step([x])
    with pytest.raises(Exception, match="lr must be finite"):
        P.AdamW([x]).step([y], lr=math.nan)
    with pytest.raises(ValueError, match=r"params\[1\] overlaps params\[0\]"):
        P.AdamW([x, x])
    with pytest.raises(ValueError, match="overlaps"):
        b = torch.zeros(256, dtype=torch.uint8, device="cuda")
        P.AdamW([b.view(F32)], copies=[b.view(BF)[:64]])
    with pytest.raises(TypeError, match=r"params\[0\]"):
        P.AdamW([x.half()])
    with pytest.raises(TypeError, match=r"copies\[0\]"):
        P.AdamW([x], copies=[y])
    with pytest.raises(ValueError, match="contiguous"):
        P.AdamW([torch.zeros(8, 8, device="cuda").t()])
    with pytest.raises(ValueError, match="2 weight_decay for 1"):
        P.AdamW([x], weight_decay=[0.0, 0.1])
    with pytest.raises(ValueError, match="states must be one of"):
        P.AdamW([x], states="4bit")
    assert int(opt.state["count"]) == 0
    empty = P.AdamW([])
    empty.step([])
    assert int(empty.state["count"]) == 1

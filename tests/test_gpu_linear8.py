"""The linear layer in 8 bits against its fp64 definition, on a GB300.

The codes and their powers of two are exact, and so are the products (eight bits of mantissa in all), so what is off is the
sums: U = 2^-24 times the sum of the products' magnitudes for each addition on a term's way.  The tensor cores
add 32 products and the accumulator in one instruction and may cut off what is below the last bit: 2 U an instruction,
depth / 32 of them, at most 128 for weight gradients, whose parts (of 4096 rows) and slices are then added one by one.
dbias: a thread adds 32 rows of each of its tiles, then quarters and parts.  bf16 outputs are rounded once, 2^-8.
"""

import numpy as np
import pytest
import torch

from oracle import train_ops_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0**-24


@pytest.fixture(scope="module")
def P():
    from co_folding_pair_gb300 import train_ops
    return train_ops


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


def inputs(g, rows, K, N, wdt=BF, spread=1.0):
    x = (randn(g, rows, K) * torch.exp(spread * randn(g, K)) * torch.exp(spread * randn(g, rows, 1))).to(BF)
    w = (randn(g, N, K) / K**0.5 * torch.exp(spread * randn(g, N, 1))).to(wdt)
    dy = (1e-3 * randn(g, rows, N) * torch.exp(spread * randn(g, N)) * torch.exp(spread * randn(g, rows, 1))).to(BF)
    return x, w, dy


def check_forward(y, x, w, b, what="y"):
    ref, mag = O.linear8(f64(x), f64(w), f64(b))
    tol = (2 * -(-x.shape[1] // 32) + 2) * U * (mag + (0 if b is None else np.abs(f64(b))))
    within(y, ref, 2.0**-8 * (np.abs(ref) + tol) + tol, what)


def check_backward(got, x, w, dy):
    rows, N = dy.shape
    (dx, dxm), (dw, dwm), (db, dbm) = O.linear8_backward(f64(x), f64(w), f64(dy))
    if got["dx"] is not None:
        tol = (2 * -(-N // 32) + 2) * U * dxm
        within(got["dx"], dx, 2.0**-8 * (np.abs(dx) + tol) + tol, "dx")
    if got["dw"] is not None:
        within(got["dw"], dw, (2 * min(128, -(-rows // 32)) + rows // 4096 + 130) * U * dwm, "dw")
        assert np.linalg.norm(f64(got["dw"]) - dw) <= 2e-6 * np.linalg.norm(dw)
    if got["dbias"] is not None:
        within(got["dbias"], db, (rows // 4 + 700) * U * dbm, "dbias")


@pytest.mark.parametrize("rows,K,N", [
    (128, 128, 128), (256, 256, 256), (1, 8, 8), (7, 24, 40), (129, 136, 72), (255, 128, 264), (257, 520, 8), (1000, 32, 128),
    (300, 1032, 776), (64, 2048, 512), (20000, 64, 32), (513, 4096, 264),
])
@pytest.mark.parametrize("wdt,bias,spread", [(BF, False, 0.0), (F32, True, 1.5)], ids=["bf16", "fp32-bias-spread"])
def test_linear8(P, rows, K, N, wdt, bias, spread):
    g = rng_of(rows + K + N)
    x, w, dy = inputs(g, rows, K, N, wdt, spread)
    b = 0.1 * randn(g, N) if bias else None
    lin = P.Linear8(w, b)
    y = lin(x, flags=P.FLAG_CHECK)
    check_forward(y, x, w, b)
    check_backward(lin.backward(x, dy, flags=P.FLAG_CHECK), x, w, dy)


@pytest.mark.parametrize("rows,K,N", [(700, 16, 4104), (40000, 256, 2056), (1, 8, 65536), (3, 65536, 16), (130, 384, 5000)])
def test_linear8_wide_with_a_bias(P, rows, K, N):
    """More outputs than a block of processors keeps biases for, and the widest layers."""
    g = rng_of(rows + N)
    x, w, dy = inputs(g, rows, K, N)
    b = randn(g, N)
    lin = P.Linear8(w, b)
    check_forward(lin(x, flags=P.FLAG_CHECK), x, w, b)
    check_backward(lin.backward(x, dy, flags=P.FLAG_CHECK), x, w, dy)


@pytest.mark.parametrize("rows,K,N", [(100003, 264, 136), (70000, 1024, 520), (4096 * 9 + 1, 8, 8)])
def test_linear8_gradients_over_many_rows(P, rows, K, N):
    """Several accumulations and slices of rows, tiles with ragged ends."""
    x, w, dy = inputs(rng_of(rows), rows, K, N, spread=0.5)
    lin = P.Linear8(w, torch.zeros(N, device="cuda"))
    check_backward(lin.backward(x, dy, flags=P.FLAG_CHECK), x, w, dy)


def test_linear8_leading_shapes_and_outputs(P):
    g = rng_of(3)
    x, w, dy = inputs(g, 6 * 35, 72, 40)
    lin = P.Linear8(w)
    flat = lin(x)
    y = torch.empty(2, 3, 35, 40, dtype=BF, device="cuda")
    assert lin(x.view(2, 3, 35, 72), out=y) is y and torch.equal(y.view(-1, 40), flat)
    ref = lin.backward(x, dy, want=("dx", "dw", "dbias"))
    dx, dw = torch.empty(2, 3, 35, 72, dtype=BF, device="cuda"), torch.empty(40, 72, device="cuda")
    got = lin.backward(x.view(2, 3, 35, 72), dy.view(2, 3, 35, 40), dx=dx, dw=dw)
    assert got["dx"] is dx and got["dw"] is dw and got["dbias"] is None
    assert torch.equal(dx.view(-1, 72), ref["dx"]) and torch.equal(dw, ref["dw"])
    for want in (("dx",), ("dw",), ("dbias",), ("dx", "dbias"), ()):
        part = lin.backward(x, dy, want=want)
        for k in ("dx", "dw", "dbias"):
            assert torch.equal(part[k], ref[k]) if k in want else part[k] is None
    assert tuple(lin(x[5]).shape) == (40,) and torch.equal(lin(x[5]), flat[5])  # one token


def test_linear8_repeats(P):
    """Bit for bit, and each row whatever the others are (one tile or another, alone or among many)."""
    x, w, dy = inputs(rng_of(4), 3000, 520, 264)
    lin = P.Linear8(w)
    y, g = lin(x), lin.backward(x, dy)
    for _ in range(3):
        assert torch.equal(lin(x), y)
        h = lin.backward(x, dy)
        assert torch.equal(h["dx"], g["dx"]) and torch.equal(h["dw"], g["dw"])
    assert torch.equal(lin(x[1000:1300].contiguous()), y[1000:1300])


@pytest.mark.parametrize("K,N", [(264, 136), (256, 264), (128, 520), (1024, 256)])
def test_linear8_repeats_many_times(P, K, N):
    """Rings that are reused thousands of times, at full speed: every pass gives the first one's bits."""
    x, w, dy = inputs(rng_of(K), 1 << 18, K, N)
    lin = P.Linear8(w)
    y, g = lin(x), lin.backward(x, dy)
    off = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        h = lin.backward(x, dy)
        off += (lin(x) != y).sum() + (h["dx"] != g["dx"]).sum() + (h["dw"] != g["dw"]).sum()
    assert int(off) == 0


@pytest.mark.parametrize("rows,K,N", [(70001, 128, 520), (300, 8, 19976), (129, 64, 136), (1, 8, 16), (513, 256, 1000),
                                      (5000, 304, 1000), (4097, 512, 264)])
def test_linear8_bias_gradient_alone_and_together(P, rows, K, N):
    """Where dy is rounded on its way to dW, its columns are added there; dbias alone has the same bits.  19976 outputs are
    more tiles than there are pairs of processors, with an odd number of blocks each."""
    x, w, dy = inputs(rng_of(rows + N), rows, K, N)
    lin = P.Linear8(w, torch.zeros(N, device="cuda"))
    every = lin.backward(x, dy, flags=P.FLAG_CHECK)
    check_backward(every, x, w, dy)
    for want in (("dbias",), ("dx", "dbias"), ("dw", "dbias")):
        part = lin.backward(x, dy, want=want, flags=P.FLAG_CHECK)
        assert all(torch.equal(part[k], every[k]) for k in want)
    again = lin.backward(x, dy)
    assert all(torch.equal(again[k], every[k]) for k in again)


def test_linear8_no_rows(P):
    w = randn(rng_of(5), 16, 24, dtype=BF)
    lin = P.Linear8(w, torch.ones(16, device="cuda"))
    x, dy = torch.empty(0, 24, dtype=BF, device="cuda"), torch.empty(0, 16, dtype=BF, device="cuda")
    assert lin(x, flags=P.FLAG_CHECK).shape == (0, 16)
    got = lin.backward(x, dy, dw=torch.ones(16, 24, device="cuda"))
    assert got["dx"].shape == (0, 24) and (got["dw"] == 0).all() and (got["dbias"] == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_linear8_keeps_what_is_not_finite_apart(P, bad):
    """A row of x with such a number gives a row of NaN, its block's other numbers keeping their rounding; in dW it reaches
    its own channel alone."""
    rows, K, N = 300, 264, 136
    x, w, dy = inputs(rng_of(6), rows, K, N)
    lin = P.Linear8(w, torch.zeros(N, device="cuda"))
    y, g = lin(x), lin.backward(x, dy)
    x2, dy2 = x.clone(), dy.clone()
    x2[17, 130] = bad
    y2 = lin(x2)
    assert torch.isnan(y2[17]).all()
    y2[17] = y[17]
    assert torch.equal(y2, y)
    g2 = lin.backward(x2, dy)
    assert torch.equal(g2["dx"], g["dx"]) and torch.isnan(g2["dw"][:, 130]).all()
    g2["dw"][:, 130] = g["dw"][:, 130]
    assert torch.equal(g2["dw"], g["dw"])
    dy2[201, 7] = bad
    g3 = lin.backward(x, dy2)
    assert torch.isnan(g3["dx"][201]).all() and torch.isnan(g3["dw"][7]).all() and not torch.isfinite(g3["dbias"][7])
    g3["dx"][201], g3["dw"][7], g3["dbias"][7] = g["dx"][201], g["dw"][7], g["dbias"][7]
    assert all(torch.equal(g3[k], g[k]) for k in g)
    w2 = w.clone()
    w2[5, 3] = bad
    lin.pack(w2)
    assert torch.isnan(lin(x)[:, 5]).all() and torch.isfinite(lin(x)[:, 6:]).all()


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e30, 3e38])
def test_linear8_of_large_and_small_values(P, size):
    """Powers of two at their ends: 2^-126 is the least, products past fp32's range overflow as fp32 does."""
    rows, K, N = 40, 136, 24
    g = rng_of(7)
    x = (randn(g, rows, K).clamp(-1, 1) * size).to(BF)
    w = randn(g, N, K, dtype=BF) if size < 1 else (randn(g, N, K) * 1e-4).to(BF)
    lin = P.Linear8(w)
    ref, mag = O.linear8(f64(x), f64(w))
    tol = (2 * 5 + 2) * U * mag + 8 * 2.0**-126  # each of eight instructions may flush a subnormal sum
    within(lin(x), ref, 2.0**-8 * (np.abs(ref) + tol) + tol, "y")
    zero = P.Linear8(torch.zeros_like(w))
    assert (zero(x) == 0).all() and (lin(torch.zeros_like(x)) == 0).all()


def test_linear8_every_code(P):
    """Products with the identity give the codes back: every bf16 number of a range, beside a block's largest one."""
    n = 128
    lin = P.Linear8(torch.eye(n, device="cuda"))  # (its power of two: 1 is 256 2^-8)
    bits = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32, device="cuda").to(torch.int16).view(BF)
    v = bits[torch.isfinite(bits)]
    v = torch.nn.functional.pad(v, (0, -v.numel() % (n - 1))).view(-1, n - 1)
    for top in (1.75, 448.0, 449.0, 1.0):
        x = torch.where(v.abs() <= top, v, 0.0)
        x = torch.cat([torch.full((len(x), 1), top, dtype=BF, device="cuda"), x], 1).contiguous()
        assert np.array_equal(f64(lin(x)), O.by_rows(f64(x)))


def test_linear8_in_a_graph_and_on_streams(P):
    """Two captured passes replayed on two streams at once, and eager calls behind work of their own stream."""
    rows, K, N = 700, 136, 264
    passes = []
    for k in range(2):
        x, w, dy = inputs(rng_of(40 + k), rows, K, N)
        lin = P.Linear8(w, torch.zeros(N, device="cuda"))
        lin.backward(x, dy), lin(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lin.pack(w)
            y, g = lin(x), lin.backward(x, dy)
        passes.append((x, w, dy, graph, y, g, lin))  # (the layer's memory is the graph's)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k, (x, w, dy, *_) in enumerate(passes):
        fresh = inputs(rng_of(50 + k), rows, K, N)
        for a, b in zip((x, w, dy), fresh):
            a.copy_(b)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, p in zip(streams, passes):
            with torch.cuda.stream(s):
                p[3].replay()
    torch.cuda.synchronize()
    for x, w, dy, _, y, g, _ in passes:
        check_forward(y, x, w, None)
        check_backward(g, x, w, dy)
    x, w, dy = (torch.zeros_like(t) for t in passes[0][:3])
    s = streams[0]
    s.wait_stream(torch.cuda.current_stream())
    lin = P.Linear8(passes[0][1], torch.zeros(N, device="cuda"))
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        for a, b in zip((x, w, dy), passes[0][:3]):
            a.copy_(b)
    y, g = lin.forward(x, stream=s), lin.backward(x, dy, stream=s)
    s.synchronize()
    check_forward(y, *passes[0][:2], None)
    check_backward(g, *passes[0][:3])


def test_linear8_small_calls_of_many_streams(P):
    """Each stream keeps the word in which its calls' kernels say that they gave up."""
    x, w, _ = inputs(rng_of(13), 300, 32, 72)
    lin = P.Linear8(w)
    want = lin(x)
    streams = [torch.cuda.Stream() for _ in range(6)]
    torch.cuda.synchronize()
    got = []
    for _ in range(50):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(lin(x))
    with pytest.raises(Exception, match="bounded wait"):  # on one of them a stall, which no other call sees
        with torch.cuda.stream(streams[2]):
            lin(x, flags=P.FLAG_CHECK | P.FLAG_INJECT_STALL)
    for s in streams:
        with torch.cuda.stream(s):
            got.append(lin(x, flags=P.FLAG_CHECK))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


def test_linear8_writes_nothing_else(P):
    """Outputs, workspaces and packed weights with bands around them."""
    from co_folding_pair_gb300 import _lib
    lib = _lib.load()
    band = 4096
    for rows, K, N in ((1, 8, 8), (129, 136, 72), (300, 24, 264)):
        x, w, dy = inputs(rng_of(60 + K), rows, K, N)
        sizes = {"packed": lib.trimul_linear8_packed_bytes(N, K), "y": rows * N * 2, "dx": rows * K * 2, "dw": N * K * 4, "db": N * 4,
                 "wf": lib.trimul_linear8_forward_workspace_bytes(rows, N, K), "wb": lib.trimul_linear8_backward_workspace_bytes(rows, N, K)}
        buf = {k: torch.full((2 * band + n + 256,), 0x5A, dtype=torch.uint8, device="cuda") for k, n in sizes.items()}
        at = {k: v.data_ptr() + band for k, v in buf.items()}
        kept = [t.clone() for t in (x, w, dy)]
        assert lib.trimul_linear8_pack(w.data_ptr(), 0, N, K, at["packed"], sizes["packed"], 0, None, 1) == 0
        assert lib.trimul_linear8_forward(at["packed"], None, x.data_ptr(), rows, N, K, at["y"], at["wf"], sizes["wf"], 0, None, 1) == 0
        assert lib.trimul_linear8_backward(at["packed"], x.data_ptr(), dy.data_ptr(), rows, N, K, at["dx"], at["dw"], at["db"], at["wb"],
                                           sizes["wb"], 0, None, 1) == 0
        torch.cuda.synchronize()
        for k, v in buf.items():
            assert (v[:band] == 0x5A).all() and (v[band + sizes[k]:] == 0x5A).all(), (k, rows)
        assert all(torch.equal(a, b) for a, b in zip(kept, (x, w, dy)))
        y = buf["y"][band:band + sizes["y"]].view(BF).view(rows, N)
        check_forward(y, x, w, None)


def test_linear8_past_32_bits(P):
    """More than 2^31 elements of x and y: the last rows."""
    rows, K, N = (1 << 31) // 256 + 300, 256, 264
    x = torch.zeros(rows, K, dtype=BF, device="cuda")
    g = rng_of(9)
    tail, w, dyt = inputs(g, 600, K, N)
    x[-600:] = tail
    lin = P.Linear8(w)
    y = lin(x, flags=P.FLAG_CHECK)
    check_forward(y[-600:], tail, w, None)
    assert (y[:-600] == 0).all()
    y.zero_()
    y[-600:] = dyt
    got = lin.backward(x, y, flags=P.FLAG_CHECK)
    first = rows - 600
    lead = first - first // 128 * 128  # blocks of 128 rows begin at multiples of 128
    pad = lambda t: torch.cat([t.new_zeros(lead, t.shape[1]), t])  # noqa: E731
    ref = lin.backward(pad(tail), pad(dyt))
    assert torch.equal(got["dx"][-600:], ref["dx"][lead:]) and (got["dx"][:-600] == 0).all()
    within(got["dw"], f64(ref["dw"]), 2 * U * 600 * np.abs(f64(dyt)).max() * np.abs(f64(tail)).max(), "dw")
    del x, y, got
    torch.cuda.empty_cache()


def test_linear8_reports_a_stalled_kernel(P):
    """Loads that never come: the waits end, the call says so, and the next one is right."""
    x, w, dy = inputs(rng_of(10), 300, 136, 72)
    lin = P.Linear8(w)
    with pytest.raises(Exception, match="bounded wait"):
        lin(x, flags=P.FLAG_CHECK | P.FLAG_INJECT_STALL)
    with pytest.raises(Exception, match="bounded wait"):
        lin.backward(x, dy, flags=P.FLAG_CHECK | P.FLAG_INJECT_STALL)
    check_forward(lin(x, flags=P.FLAG_CHECK), x, w, None)
    check_backward(lin.backward(x, dy, flags=P.FLAG_CHECK), x, w, dy)


def test_linear8_refusals(P):
    g = rng_of(11)
    x, w, dy = inputs(g, 32, 24, 16)
    lin = P.Linear8(w)
    with pytest.raises(ValueError, match="x must be"):
        lin(x[:, :16].contiguous())
    with pytest.raises(ValueError, match="contiguous"):
        lin(torch.zeros(24, 32, dtype=BF, device="cuda").t())
    with pytest.raises(TypeError, match="x must be"):
        lin(x.float())
    with pytest.raises(ValueError, match="dy must be"):
        lin.backward(x, dy[:8].contiguous())
    with pytest.raises(ValueError, match="unknown gradient"):
        lin.backward(x, dy, want=("dz",))
    with pytest.raises(ValueError, match="out must be"):
        lin(x, out=torch.empty(32, 24, dtype=BF, device="cuda"))
    with pytest.raises(ValueError, match="weight must be"):
        lin.pack(w[:8].contiguous())
    with pytest.raises(ValueError, match="bias must be"):
        P.Linear8(w, torch.zeros(24, device="cuda"))
    with pytest.raises(TypeError, match="weight"):
        P.Linear8(w.half())
    with pytest.raises(Exception, match="multiples of 8"):
        P.Linear8(torch.zeros(12, 24, dtype=BF, device="cuda"))
    with pytest.raises(Exception, match="dx overlaps x"):
        lin.backward(x, dy, dx=x)
    with pytest.raises(Exception, match="16-byte aligned"):
        lin(torch.zeros(32 * 24 + 1, dtype=BF, device="cuda")[1:].view(32, 24))


def test_linear8_refuses_a_buffer_for_what_is_not_wanted(P):
    """It would be left as it is."""
    g = rng_of(12)
    x, w, dy = inputs(g, 32, 24, 16)
    lin, db = P.Linear8(w), torch.empty(16, device="cuda")
    with pytest.raises(ValueError, match="dbias is given but not among"):
        lin.backward(x, dy, dbias=db)
    with pytest.raises(ValueError, match="dw is given but not among"):
        lin.backward(x, dy, dw=torch.empty(16, 24, device="cuda"), want=("dx",))
    got = lin.backward(x, dy, dbias=db, want=("dbias",))
    assert got["dbias"] is db and got["dx"] is None and got["dw"] is None
    check_backward(got, x, w, dy)

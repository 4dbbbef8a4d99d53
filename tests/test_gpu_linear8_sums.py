"""Sums of the linear layer in 8 bits over many rows, on a GB300: whole numbers, whose sums are exact whatever their order, and
dbias within the additions that it takes.

Additions on a term's way to dbias, U = 2^-24 of the sum of magnitudes each.  Where dy is rounded on its way to dW (fewer
channels in than out, 512 of them at most), a lane adds 8 rows of every other block of a slice, then 4 joins its lanes and two sums
a slice are joined, each eighth by one thread: 8 ceil(per_z / 2) + 4 + 2 n_z / 8 + 8.  Else a thread adds 8 rows of each of its
tiles, one joins two lanes, 8 the warps, and the parts are joined likewise: 8 ceil(tiles / parts) + 9 + parts / 8 + 8.  The
counts below take at least 64 pairs and 128 processors, and at most 128 and 256.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0**-24


@pytest.fixture(scope="module")
def P():
    from co_folding_pair_gb300 import train_ops
    return train_ops


def rng_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def up(a, b):
    return -(-a // b)


def additions(rows, K, N):
    tiles = up(rows, 128)
    if K < N and K <= 512:
        n = max(1, min(up(tiles, 4), 64 // (up(N, 256) * up(K, 256))))
        return 8 * up(4 * up(up(tiles, n), 4), 2) + 4 + 2 * 128 // 8 + 8
    parts = max(1, min(tiles, 3 * 128 // up(N, 128)))
    return 8 * up(tiles, parts) + 9 + 3 * 256 // 8 + 8


SHAPES = [(100003, 264, 136), (100003, 136, 264), (70000, 1024, 520), (70000, 520, 1024), (300001, 8, 16), (300001, 16, 8), (4097, 640, 768),
          (1 << 19, 128, 512), (200000, 512, 520), (131, 8, 65536)]


@pytest.mark.parametrize("rows,K,N", SHAPES)
def test_whole_numbers_are_exact(P, rows, K, N):
    """Codes, products and sums below 2^24 are exact: a row that is missing or taken twice shows, wherever it is."""
    g = rng_of(rows + N)
    whole = lambda most, *shape: torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(F32)  # noqa: E731
    x, w, dy, b = whole(3, rows, K), whole(2, N, K), whole(4, rows, N), whole(100, N)
    lin = P.Linear8(w, b)
    y, got = lin(x.to(BF), flags=P.FLAG_CHECK), lin.backward(x.to(BF), dy.to(BF), flags=P.FLAG_CHECK)
    for t, ref in ((got["dw"], dy.double().t() @ x.double()), (got["dbias"], dy.double().sum(0))):
        assert float(ref.abs().max()) < 1 << 24 and torch.equal(t.double(), ref)
    for c in range(0, rows, 1 << 16):
        at = slice(c, c + (1 << 16))
        assert torch.equal(y[at], (x[at].double() @ w.double().t() + b.double()).to(F32).to(BF))
        assert torch.equal(got["dx"][at], (dy[at].double() @ w.double()).to(F32).to(BF))
    alone = lin.backward(x.to(BF), dy.to(BF), want=("dbias",), flags=P.FLAG_CHECK)
    assert torch.equal(alone["dbias"], got["dbias"])


@pytest.mark.parametrize("rows,K,N", SHAPES)
def test_dbias_within_its_additions(P, rows, K, N):
    g = rng_of(rows + K)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    x, dy = randn(rows, K).to(BF), (randn(rows, N) * torch.exp(randn(rows, 1)) + 0.1).to(BF)
    got = P.Linear8(randn(N, K), randn(N)).backward(x, dy, want=("dbias",), flags=P.FLAG_CHECK)["dbias"].double()
    ref, mag = dy.double().sum(0), dy.double().abs().sum(0)
    assert bool(((got - ref).abs() <= additions(rows, K, N) * U * mag).all())


@pytest.mark.parametrize("K,N", [(128, 1000), (1000, 128), (264, 520), (520, 264)])
def test_a_row_is_the_same_among_few_and_many(P, K, N):
    """Bit for bit, on both sides of the number of rows at which another kernel takes over."""
    g = rng_of(K)
    x, w, dy = (torch.randn(*s, generator=g, device="cuda").to(BF) for s in ((70000, K), (N, K), (70000, N)))
    lin = P.Linear8(w, torch.randn(N, generator=g, device="cuda"))
    y, dx = lin(x), lin.backward(x, dy, want=("dx",))["dx"]
    for at in (slice(1000, 1300), slice(65000, 65001), slice(0, 65535)):
        few, dfew = x[at].contiguous(), dy[at].contiguous()
        assert torch.equal(lin(few), y[at])
        assert torch.equal(lin.backward(few, dfew, want=("dx",))["dx"], dx[at])

"""The definitions of oracle/train_ops_oracle.py against other statements of the same things."""

import numpy as np
import torch

from oracle import train_ops_oracle as O


def test_e4m3_is_the_formats():
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
    table = table[torch.isfinite(table)].numpy()
    assert (O.e4m3(table) == table).all() and table.max() == 448
    y = np.concatenate([np.linspace(-460, 460, 20011), np.linspace(-0.1, 0.1, 20011), (table[:-1] + table[1:]) / 2])
    y32 = np.clip(y.astype(np.float32), -448, 448)
    want = torch.from_numpy(y32).to(torch.float8_e4m3fn).float().numpy()
    assert (O.e4m3(y32.astype(np.float64)) == want).all()


def test_random_rounding_is_to_the_neighbours():
    y = np.concatenate([np.linspace(-447, 447, 5001), np.linspace(-0.05, 0.05, 5001)])
    lo, hi = O.e4m3_at_random(y, 0.0), O.e4m3_at_random(y, 1 - 2.0**-16)
    assert (np.abs(lo) <= np.abs(y)).all() and (np.abs(hi) >= np.abs(y) - O._step(y) * 2.0**-15).all()
    assert (O.e4m3(lo) == lo).all() and (O.e4m3(hi) == hi).all()
    mean = np.mean([O.e4m3_at_random(y, (k + 0.5) / 1024) for k in range(1024)], axis=0)
    assert (np.abs(mean - y) <= O._step(y) / 1024).all()


def test_hash_is_spread():
    h = O.random_bits(3, 5, 2, np.arange(1 << 16))
    assert len(np.unique(h)) > 65000
    for s in range(32):  # each bit is one half of the time, within 6 deviations
        assert abs(float(np.mean(h >> np.uint64(s) & np.uint64(1))) - 0.5) <= 6 * 0.5 / 256
    assert (O.random_bits(3, 5, 2, np.arange(8)) != O.random_bits(3, 6, 2, np.arange(8))).all()


def test_adamw_is_torchs():
    rng = np.random.default_rng(0)
    p = rng.standard_normal(50)
    t = torch.nn.Parameter(torch.from_numpy(p.copy()))
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    m, v = np.zeros(50), np.zeros(50)
    for k in range(1, 6):
        g = rng.standard_normal(50)
        t.grad = torch.from_numpy(g)
        opt.step()
        p, m, v, *_ = O.adamw(p, g, m, v, k, 1e-2, (0.8, 0.95), 1e-6, 0.1)
        assert np.allclose(t.detach().numpy(), p, rtol=1e-13, atol=1e-14)


def test_quantized_by_another_statement():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((70, 300)) * np.exp(rng.standard_normal((70, 300)))
    q = O.by_rows(x)
    for r in range(70):
        for b in range(0, 300, 128):
            v = x[r, b:b + 128]
            e = -126
            while np.abs(v).max() > 448 * 2.0**e:
                e += 1
            assert (q[r, b:b + 128] == O.e4m3(v * 2.0**-e) * 2.0**e).all()
    assert (O.by_columns(x) == O.by_rows(x.T).T).all()
    w = rng.standard_normal((130, 140))
    p = O.by_blocks(w)
    assert (O.by_blocks(w.T) == p.T).all() and np.abs(p - w).max() <= 2.0**-4 * np.abs(w).max()
    assert (O.quantized(np.array([448.0, -3.0]), 0) == [448, -3]).all() and (O.quantized(np.array([449.0, 9.0]), 0) == [448, 9]).all()
    assert (O.quantized(np.zeros(4), 0) == 0).all()
    bad = O.quantized(np.array([np.inf, 1.0625, np.nan, 2.0]), 0)
    assert np.isnan(bad[[0, 2]]).all() and (bad[[1, 3]] == O.quantized(np.array([1.0625, 2.0]), 0)).all()


def test_linear8_gradients_are_the_products_derivatives():
    """With operands that 8 bits hold, rounding changes nothing and dx, dW, dbias are those of x W^T + b."""
    rng = np.random.default_rng(2)
    x, w, dy = (rng.integers(-8, 9, s).astype(np.float64) for s in ((40, 24), (16, 24), (40, 16)))
    b = np.ones(16)
    (dx, _), (dw, _), (db, _) = O.linear8_backward(x, w, dy)
    f = lambda x, w, b: float((O.linear8(x, w, b)[0] * dy).sum())  # noqa: E731
    assert (O.linear8(x, w, b)[0] == x @ w.T + b).all()
    for t, d in ((x, dx), (w, dw), (b, db)):
        for i in range(0, t.size, 37):
            u = t.copy()
            u.flat[i] += 1 if u.flat[i] < 8 else -1
            args = [u if s is t else s for s in (x, w, b)]
            assert f(*args) - f(x, w, b) == (u.flat[i] - t.flat[i]) * d.flat[i]

"""fp64 CPU definitions of AdamW and of the linear layer in 8 bits.

Plain numpy, written from the definitions in include/trimul.h.  test_oracle_train_ops.py
holds them against differences, torch's own AdamW and tables of the formats.
"""

import math

import numpy as np

BLOCK = 128


# ------------------------------------------------------------------ e4m3
def _step(y):
    """How far apart the e4m3 numbers around |y| are."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0**-6))) - 3)


def e4m3(y):
    """y to the nearest e4m3 number, ties to even, values past 448 to 448."""
    s = _step(y)
    return np.clip(np.round(y / s) * s, -448.0, 448.0)


def e4m3_at_random(y, chance):
    """One of the two neighbours of y: the upper one (in magnitude) where y's place between them and chance pass 1."""
    s = _step(y)
    return np.sign(y) * np.minimum(np.floor(np.abs(y) / s + chance) * s, 448.0)


# ------------------------------------------------------------------ random bits
def pcg(x):
    """The PCG hash of Jarzynski and Olano (2020), of 32-bit whole numbers."""
    x = np.asarray(x, dtype=np.uint64) & np.uint64(0xFFFFFFFF)
    mask = np.uint64(0xFFFFFFFF)
    x = (x * np.uint64(747796405) + np.uint64(2891336453)) & mask
    x = (((x >> ((x >> np.uint64(28)) + np.uint64(4))) ^ x) * np.uint64(277803737)) & mask
    return (x >> np.uint64(22)) ^ x


def random_bits(seed, t, tensor, index):
    """32 bits for each element (its index) of a tensor (its place in the call) at step t."""
    key = pcg(pcg(np.uint64(tensor) + pcg(np.uint64(t) + pcg(np.uint64(seed)))) + (np.asarray(index, np.uint64) >> np.uint64(32)))
    return pcg(key ^ (np.asarray(index, np.uint64) & np.uint64(0xFFFFFFFF)))


def bf16_at_random(p, bits16):
    s = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(p), 2.0**-126))) - 7)
    return np.sign(p) * np.floor(np.abs(p) / s + bits16 / 65536.0) * s


# ------------------------------------------------------------------ AdamW
def clip_factor(norm, max_norm):
    return 1.0 if norm is None else min(1.0, max_norm / (norm + 1e-6))


def adamw(p, g, m, v, t, lr, betas, eps, decay, clip=1.0):
    """The new p, m, v, and the magnitudes that the errors of m, v and p's step are measured by."""
    b1, b2 = betas
    g = clip * g
    m, mag = b1 * m + (1 - b1) * g, b1 * np.abs(m) + (1 - b1) * np.abs(g)
    v = b2 * v + (1 - b2) * g * g
    den = np.sqrt(v / (1 - b2**t)) + eps
    rate = lr / (1 - b1**t)
    return p - lr * decay * p - rate * m / den, m, v, mag, abs(rate) * mag / den


def blocks(x):
    """x as rows of 128, zeros behind its end."""
    return np.pad(x, (0, -len(x) % BLOCK)).reshape(-1, BLOCK)


def scales(x):
    return np.maximum(np.abs(blocks(x)).max(1), 2.0**-90) / 448


def dequantized(codes, scale):
    return codes * np.repeat(scale, BLOCK)[: len(codes)]


# ------------------------------------------------------------------ linear layer in 8 bits
def quantized(v, axes):
    """Q(v) for blocks along `axes` of an array, what is not finite as NaN."""
    fine = np.isfinite(v)
    a = np.where(fine, np.abs(v), 0.0).max(axis=axes, keepdims=True)
    e = np.maximum(np.ceil(np.log2(np.maximum(a, 2.0**-200) / 448)), -126)  # (a quotient that is a power of two is exact)
    return np.where(fine, e4m3(np.where(fine, v, 0.0) * 2.0**-e) * 2.0**e, np.nan)


def _tiles(x, down, along):
    R, C = x.shape
    return np.pad(x, ((0, -R % down), (0, -C % along))).reshape(-(-R // down), down, -(-C // along), along)


def by_rows(x):
    return quantized(_tiles(x, 1, BLOCK), 3).reshape(x.shape[0], -1)[:, : x.shape[1]]


def by_columns(x):
    return quantized(_tiles(x, BLOCK, 1), 1).reshape(-1, x.shape[1])[: x.shape[0]]


def by_blocks(w):
    N, K = w.shape
    return quantized(_tiles(w, BLOCK, BLOCK), (1, 3)).reshape(N + -N % BLOCK, -1)[:N, :K]


def linear8(x, w, bias=None):
    """y before its rounding, and the sums of the products' magnitudes."""
    q, p = by_rows(x), by_blocks(w)
    y = q @ p.T
    return (y if bias is None else y + bias), np.abs(q) @ np.abs(p).T


def linear8_backward(x, w, dy):
    """dx (before its rounding), dW, dbias, each with its products' magnitudes."""
    r, p = by_rows(dy), by_blocks(w)
    c, d = by_columns(dy), by_columns(x)
    return (r @ p, np.abs(r) @ np.abs(p)), (c.T @ d, np.abs(c).T @ np.abs(d)), (dy.sum(0), np.abs(dy).sum(0))

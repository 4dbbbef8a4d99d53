"""The bounds that the residual step's gradients are held to as whole tensors.

U = 2^-24.  Element by element, a bound has to allow for the worst row; the
2-norm of a tensor's error against its own does not, and so sees what an
element's bound hides: a missing term of a derivative, a wrong factor, a sum
that is not there.

- Rounding to bf16 is at most 2^-8 of each element, so at most 2^-8 of the norm;
  to fp32 it is U.
- Before it come some twenty fp32 operations and sums of up to 256 terms over a
  tree of at most 13 levels, twice, each off by U (the reciprocal square roots
  by 4 U) of the numbers that they work on: within 64 U of these.  They are the
  terms of the derivative, whose norms for the inputs here (values near 1,
  deviations near 1) are at most four times the result's: 256 U = 2^-16.
- A parameter's gradient is a column sum.  Its terms are off by 256 U as above,
  and each addition on a term's way by U of a partial sum, at most the sum of
  the magnitudes: (256 + 4 adds) U of the norm of these sums, where the way is
  a thread's rows, a block's rows, 32 groups of blocks and a tree of five.
"""

import numpy as np

U = 2.0**-24
INNER = 256 * U
SHARE = 0.05  # of a gradient's norm: no bound may be more, so that none accepts zeros


def lanes(D):
    g = 1
    while g * 8 < D:
        g *= 2
    return g


def additions(rows, D, blocks=304):
    """The most additions that a term of a column sum goes through (`blocks`: resident at once)."""
    per_block = 256 // lanes(D)
    n = min(blocks, -(-rows // per_block))
    return -(-rows // (n * per_block)) + per_block + -(-n // 32) + 5


def bound(name, ref, mag=None, bf16=True, rows=0):
    """The most that the 2-norm of a tensor's error may be; mag: the sums of a parameter's terms' magnitudes."""
    if mag is None:
        return ((2.0**-8 if bf16 else U) + INNER) * np.linalg.norm(ref)
    D = ref.shape[-1]
    return (256 + 4 * additions(rows, D)) * U * np.linalg.norm(mag)


def off(got, ref, limit):
    """The error's 2-norm as a share of the limit; infinite where something is not finite."""
    err = np.linalg.norm(np.asarray(got, dtype=np.float64) - ref)
    return np.inf if not np.isfinite(err) else err / limit if limit > 0 else (0.0 if err == 0 else np.inf)

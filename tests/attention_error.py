"""What the rounding of attention outputs may come to, by its root mean square.

A bound on the largest error has to add up what every position could
contribute, and is wide for long sequences.  Roundings of different positions
are independent, so their sum is held here by its root mean square instead:
the output's own rounding to bfloat16, uniform within half a step, and the
arithmetic's part.  A low part of the weights that is missing doubles the mean
square; one missing or wrongly scaled part of a long sequence is many steps.
"""

import numpy as np

F32 = 2.0 ** -24


def softmax_moments(q, k, v, scale):
    """(out, lse, weighted, spread) of queries q [G, D] over keys and values [L, D], float64.

    weighted: sqrt(sum p^2 v^2) / sum p; spread: sqrt(sum p^2 (v - out)^2) / sum p.
    """
    s = scale * (q @ k.T)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(-1, keepdims=True)
    p /= total
    out = p @ v
    square = p * p
    weighted = square @ (v * v)
    spread = weighted - 2 * out * (square @ v) + out * out * square.sum(-1, keepdims=True)
    return out, (top + np.log(total))[:, 0], np.sqrt(weighted), np.sqrt(np.maximum(spread, 0.0))


def allowed_square(out, weighted, spread, score, weight):
    """Mean square error that each output of `out` may have.

    A score's error, at most `score`, moves the output by p (v - out) of it; a
    weight's, at most `weight` of it, by p v; sums and the division pass fewer
    than 64 roundings of 2^-24 of the output where no partial sum is larger than it, and
    eight times that where they are.
    """
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(out), 1e-30))) - 7)
    return step ** 2 / 12 + (weight * weighted) ** 2 + (score * spread) ** 2 + (512 * F32 * np.abs(out)) ** 2


def assert_rms(got, out, weighted, spread, score, weight, what):
    """got and out [..., D]; all outputs together within 10 %, every row within a factor of two.

    The mean square of n such errors scatters by sqrt(4 / n) of itself (kurtosis 5: uniform, of steps that vary):
    8192 outputs are within 10 % of the root by nine deviations, a row of 64 within a factor of two by twelve.
    """
    assert got.size >= 8192
    square, allowed = (got - out) ** 2, allowed_square(out, weighted, spread, score, weight)
    ratio = np.sqrt(square.mean() / allowed.mean())
    rows = np.sqrt(square.mean(-1) / allowed.mean(-1))
    assert ratio <= 1.1 and rows.max() <= 2.0, (
        f"{what}: root mean square error {ratio:.3f} of what rounding explains, {rows.max():.3f} in one row")

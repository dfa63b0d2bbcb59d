"""Tolerances of the tests of rounded outputs.

An output is the float32 result rounded once to its type: half a step of that
type relative to the value, plus the error of the float32 arithmetic, which
each test derives and passes in.
"""

import numpy as np
import torch

F32 = 2.0 ** -24  # half a step of float32, relative


def to_np(t):
    return t.detach().to("cpu").to(torch.float64).numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def assert_rounded(got, ref, arithmetic, what):
    """|got - ref| <= half a step of got's type * |ref| + arithmetic (elementwise or a number).

    The rounded value is the float32 result, itself off by `arithmetic`, so
    that error is counted once more with the step's factor, (1 + half step).
    """
    h = half_step(got.dtype)
    g = to_np(got)
    tol = h * np.abs(ref) + (1.0 + h) * arithmetic
    err = np.abs(g - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} values off, worst error {np.nanmax(err):.3e} "
                           f"with {np.broadcast_to(tol, err.shape).flat[np.nanargmax(np.where(bad, err, -1))]:.3e} allowed")

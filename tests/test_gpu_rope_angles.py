"""Angles of kda_rope_append: sines and cosines at near and far positions, to float32's own precision."""

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from tests.rounding import F32, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def turns(steps, positions):
    """Fractions of a turn, exact to float64: position * step modulo 2^64 in integers."""
    words = steps.cpu().numpy().view(np.uint32).astype(object)
    full = [int(hi) << 32 | int(lo) for lo, hi in words]
    return np.array([[(p * s % 2 ** 64) / 2.0 ** 64 for s in full] for p in positions])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("highest", [100, 10 ** 6, 2 ** 31 - 2])
def test_cosines_and_sines(interleaved, highest):
    g = torch.Generator().manual_seed(highest % 1000)
    N, D = 2000, 128
    positions = torch.randint(0, highest + 1, (N,), generator=g)
    positions[0], positions[1] = 0, highest
    q = torch.zeros(N, 1, D, device="cuda")
    q.view(N, D // 2, 2)[:, :, 0] = 1.0
    if not interleaved:
        q.zero_()
        q[:, :, :D // 2] = 1.0
    steps = binding.kda_rope_phase_steps(D)
    pages = torch.zeros(2, 4, 1, D, device="cuda")
    out = binding.kda_rope_append(q, q, q, steps, (positions + 1).to(torch.int32).cuda(),
                                  torch.zeros(N, 1, dtype=torch.int32, device="cuda"), pages, torch.zeros_like(pages),
                                  interleaved=interleaved)
    torch.cuda.synchronize()
    got = to_np(out)[:, 0]
    cos, sin = (got[:, 0::2], got[:, 1::2]) if interleaved else (got[:, :D // 2], got[:, D // 2:])
    angle = 2 * np.pi * turns(steps, positions.tolist())
    # The function is off by at most a unit in the last place, 2^-24 below 1; its argument, an eighth of a turn at most,
    # by half a step of float32, pi 2^-27 of the angle, and by what the phase's lower half holds, pi 2^-32.
    allowed = F32 + np.pi * 2.0 ** -27 + np.pi * 2.0 ** -32 + 1e-12
    assert np.abs(cos - np.cos(angle)).max() <= allowed and np.abs(sin - np.sin(angle)).max() <= allowed

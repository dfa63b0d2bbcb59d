"""kda_prefix_attention_decode against kda_paged_attention_decode over random shapes: groups of every size, prefixes from
nothing to many tiles, short units that crowd a block and long ones over many, windows, page sizes, heads, channels."""

import random

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from tests.rounding import F32, to_np
from tests.test_gpu_paged_attention import same, tolerances
from tests.test_gpu_prefix_attention import BF16, FP32, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def draw(r):
    """Groups and the other arguments of make, with some 2^27 products of queries and keys at most."""
    while True:
        D, (Hq, Hkv), dtype = r.choice([64, 128, 256]), r.choice([(32, 8), (16, 16), (24, 8), (12, 1), (32, 2), (8, 8), (4, 1)]), \
            r.choice([BF16, BF16, BF16, FP32])
        if dtype == FP32 and (Hq // Hkv > 4 or D > 128):
            continue
        most, top = r.choice([1, 3, 7, 20, 60, 150]), r.choice([3, 70, 140, 260, 600, 2500])
        tail, crowd = r.choice([1, 20, 300]), r.choice([1, 2, 4, 9, 40])
        groups = [(r.choice([0, 1, 64, 128, top, r.randint(1, top), r.randint(1, top)]),
                   [r.randint(0 if r.random() < .1 else 1, tail) for _ in range(r.randint(0 if most > 3 else 2, crowd + 1))])
                  for _ in range(most)]
        lens = [p + t for p, tails in groups for t in tails]
        if len(lens) > len(groups) and sum(lens) * Hq * D <= 1 << 27 and sum(lens) * Hkv * D <= 1 << 25:
            return groups, dict(Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, page=r.choice([1, 7, 8, 16, 24, 32, 64, 256]))


@pytest.mark.parametrize("seed", range(60))
def test_shared_and_alone_agree(seed):
    r = random.Random(seed)
    groups, kw = draw(r)
    c = make(groups, seed=seed, **kw)
    for window in (0, r.choice([1, 50, 10 ** 6, max(c["lens"].tolist()) - 5])):
        window = max(0, window)
        out, lse = run(c, window=window)
        again, sums = run(c, window=window)
        alone, alone_sums = binding.kda_paged_attention_decode(c["q"], c["k"], c["v"], c["table"], c["lens"], window=window,
                                                               return_lse=True)
        torch.cuda.synchronize()
        assert binding.kda_device_error() == 0
        assert same(out, again) and same(lse, sums)
        empty = to_np(alone_sums) == -np.inf
        assert np.array_equal(to_np(lse) == -np.inf, empty)
        # each side is within the arithmetic's error and its own rounding of the definition
        t_out, t_lse = tolerances(c, kw["D"] ** -0.5)
        a, b = to_np(out), to_np(alone)
        assert np.all(np.abs(a - b) <= 2 * t_out + 2 * 2.0 ** -8 * (np.maximum(np.abs(a), np.abs(b)) + t_out)), (groups, kw, window)
        a, b = to_np(lse)[~empty], to_np(alone_sums)[~empty]
        assert np.all(np.abs(a - b) <= 2 * t_lse + 2 * F32 * np.maximum(np.abs(a), np.abs(b))), (groups, kw, window)

"""Log-sums of kda_beam_select: beams whose pieces are summed in different ways, and sums held to their stated error."""

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from tests.test_gpu_beam_select import check

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


LIMIT = 726817.5  # 2^20 / log2(e): from here on a piece's reference is found in float64


def two_pieces(low, high):
    """Beams with one logit at the start and one at the end of a long row, all others none; [36, 2, V] float32."""
    x = torch.full((36, 2, 40000), -float("inf"))
    x[:, :, 5], x[:, :, -3] = low.view(36, 2), high.view(36, 2)
    return x.cuda()


@pytest.mark.parametrize("step", [0.0, 0.0625, 0.5, 1.5])
@pytest.mark.parametrize("swapped", [False, True])
def test_pieces_on_either_side_of_the_limit(step, swapped):
    # every float32 of the last 4.5 below the limit: its product with log2(e) rounds to 2^-4 there, to either side of
    # an integer; beside a piece at or past the limit
    low = (LIMIT - 0.0625 * (1 + torch.arange(72, dtype=torch.float64))).float()
    high = torch.full((72,), LIMIT + step)
    x = two_pieces(high, low) if swapped else two_pieces(low, high)
    check(x, torch.randn(36, 2, generator=torch.Generator().manual_seed(1)).cuda(), 4)


@pytest.mark.parametrize("step", [0.0, 0.0625, 0.5])
def test_pieces_on_either_side_of_the_negative_limit(step):
    high = (-LIMIT + 0.125 * (1 + torch.arange(72, dtype=torch.float64))).float()
    low = torch.full((72,), -LIMIT - step)
    check(two_pieces(low, high), torch.randn(36, 2, generator=torch.Generator().manual_seed(2)).cuda(), 4)


def test_full_rows_around_the_limit():
    # what float32 can hold there: logits 1/16 apart, all pieces near their common maximum
    g = torch.Generator().manual_seed(3)
    x = LIMIT + torch.randint(-160, 33, (4, 3, 50257), generator=g).double() / 16
    check(x.float().cuda(), torch.randn(4, 3, generator=g).cuda(), 8)
    check((-x).float().cuda(), torch.randn(4, 3, generator=g).cuda(), 8)

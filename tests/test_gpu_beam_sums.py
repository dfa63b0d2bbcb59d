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


@pytest.mark.parametrize("top", [1e6, 1e20, 3e38, -1e6, -1e20, -3e38])
def test_pieces_far_past_the_limit(top):
    x = torch.full((2, 2, 30000), top)
    x[0, 0, 100], x[0, 1, 29000] = 5.0, -7.0   # above or far below the rest
    scores = torch.zeros(2, 2, device="cuda")
    if top > -1e16:
        check(x.cuda(), scores, 6)
        return
    # Exactly: beams 0 and 1 are certain of tokens 100 and 29000, and their other tokens are worth top - 5 and top + 7.
    # float64, which the oracle computes in, holds neither apart from top; the sums of two float32 do.
    got = binding.kda_beam_select(x.cuda(), scores, 6)
    assert got[1].tolist() == [[0, 1, 1, 1, 1, 1], [0] * 6]
    assert got[2].tolist() == [[100, 29000, 0, 1, 2, 3], list(range(6))]
    assert torch.equal(got[0][0].cpu(), torch.tensor([0.0, 0.0] + [top] * 4))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_forced_token_leaves_the_score_as_it_is(dtype):
    # one token allowed: its probability is 1, so equal scores tie to the lower beam and are returned to the bit
    g = torch.Generator().manual_seed(4)
    x = torch.full((64, 4, 5000), -float("inf"))
    at = torch.randint(0, 5000, (64, 4, 1), generator=g)
    x.scatter_(2, at, torch.randn(64, 4, 1, generator=g) * 30)
    s = (torch.randn(64, 1, generator=g) - 10).expand(64, 4).contiguous()
    got = check(x.to(dtype).cuda(), s.cuda(), 4)
    assert torch.equal(got[0].cpu(), s) and torch.equal(got[1].cpu(), torch.arange(4, dtype=torch.int32).expand(64, 4))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N,B,V,M", [(1, 4, 501, 4), (2, 3, 2049, 9), (3, 8, 4097, 16), (1, 32, 9001, 64), (4, 5, 50257, 5),
                                     (1, 2, 131071, 2), (40, 4, 30522, 8), (64, 3, 100003, 6)])
def test_equal_beams_tie_to_the_first_wherever_their_rows_start(dtype, N, B, V, M):
    # odd vocabularies: no two of a request's rows start alike on 16-byte boundaries
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(N, 1, V, generator=g) * 2.5).to(dtype).expand(N, B, V).contiguous().cuda()
    s = (torch.randn(N, 1, generator=g) - 10).expand(N, B).contiguous().cuda()
    check(x, s, M)  # a bfloat16 row may hold its largest logit twice: both of the first beam, then the next one's


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [777, 20001, 140001])
def test_rows_that_start_elsewhere_have_the_same_sums(dtype, V):
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(2, 3, V, generator=g) * 2.5).to(dtype).cuda()
    s = torch.randn(2, 3, generator=g).cuda()
    results = []
    for start in range(1, 8):
        wide = torch.zeros(2 * 3 * (V + 8), dtype=dtype, device="cuda")
        rows = torch.as_strided(wide, (2, 3, V), (3 * (V + 8), V + 3, 1), start)
        rows.copy_(x)
        results.append(check(rows, s, 12))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))


def log_sum_errors(x):
    """Error of the log-sums of rows x [N, 1, V], from scores that put the results near 0, where float32 is fine."""
    ref = torch.logsumexp(x.double(), -1) - x.double().amax(-1)
    s = ref.float()
    got = binding.kda_beam_select(x, s, 1)
    torch.cuda.synchronize()
    return got[0][:, 0].double() - (s.double() - ref)[:, 0]


def log_sum_error(x):
    return log_sum_errors(x).abs().max().item()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [65536, 131071])
def test_log_sums_of_constant_rows(dtype, V):
    # Every exponential has the same error, 2^-22 at most, and its argument, within 1 of 0, two roundings of 2^-25;
    # equal terms add up in a tree with one rounding at most of three of them; the rest is carried along.
    x = torch.linspace(-20, 20, 512).to(dtype).cuda().view(-1, 1, 1)
    for rows in x.split(128):
        assert log_sum_error(rows.expand(-1, 1, V).contiguous()) <= 2.0 ** -22 + 0.7 * 2.0 ** -24 + 2.0 ** -24 + 1e-9


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [65536, 131071])
@pytest.mark.parametrize("below", [1.0, 4.0, 5.5, 5.59, 11.0])
def test_log_sums_of_few_distinct_values(dtype, V, below):
    # most logits `below` the largest one, one in 256 (a thread's share) the largest: 2^-22 of the exponential, 4.4e-7 of
    # its argument's roundings (their worst, at 8 ln 2 = 5.55), six roundings of 2^-24
    top = torch.linspace(-3, 3, 96).to(dtype)
    x = (top - torch.tensor(below).to(dtype)).view(-1, 1, 1).expand(-1, 1, V).contiguous()
    x[:, 0, ::256] = top[:, None]
    assert log_sum_error(x.cuda()) <= 1.1e-6


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_log_sums_of_unequal_logits_average_out(dtype):
    # Of 65537 terms: 2^-22 bounds what the exponentials have in common, 2^-21 / sqrt(the number that weighs, over 4096)
    # the deviation of the rest, of which ten are allowed between the rows.
    g = torch.Generator().manual_seed(6)
    x = torch.randn(64, 1, 65537, generator=g).to(dtype).cuda()
    errors = log_sum_errors(x)
    assert errors.abs().max() <= 2.0 ** -22 + 10 * 2.0 ** -27 and errors.max() - errors.min() <= 10 * 2.0 ** -27


def test_log_sums_past_the_limit():
    # each term is found from its distance to the largest logit, and every addition carries its rounding
    g = torch.Generator().manual_seed(7)
    x = (LIMIT + 100 + torch.randint(0, 16, (16, 1, 70001), generator=g).double() / 16).float()
    assert log_sum_error(x.cuda()) <= 1.1e-6
    assert log_sum_error(torch.full((4, 1, 70001), 1e7, device="cuda")) <= 1.1e-6

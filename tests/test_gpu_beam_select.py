"""GPU parity of kda_beam_select against the float64 oracle: exact parents and
tokens, ties, masked logits, dead and finished beams, odd vocabularies and rows
that start anywhere, and repeated use."""

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from oracle import cache_oracle as co
from tests.rounding import F32, to_np

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def make(N, B, V, dtype=BF16, seed=0, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(N, B, V, generator=g) * spread).to(dtype).cuda()
    s = (torch.randn(N, B, generator=g) * 1.5 - 10.0).cuda()
    return x, s


def check(x, s, M, finished=None, eos=0, **kw):
    f = None if finished is None else torch.tensor(finished, dtype=torch.int32).cuda()
    got = binding.kda_beam_select(x, s, M, finished=f, eos_token=eos, **kw)
    torch.cuda.synchronize()
    ref = co.beam_select(to_np(x), to_np(s), M, finished=None if f is None else f.cpu().numpy(), eos_token=eos)
    assert np.array_equal(got[1].cpu().numpy(), ref[1]), "parents"
    assert np.array_equal(got[2].cpu().numpy(), ref[2]), "tokens"
    have = ref[1] >= 0
    out = to_np(got[0])
    assert np.all(out[~have] == -np.inf)
    # One rounding to float32, and the log-sum: each exponential is off by at most 4 half steps and its argument's
    # rounding, 2^-24 of at most 100 in the terms that matter; a thread adds 32 of them.  2^-16 bounds all of it.
    assert np.all(np.abs(out[have] - ref[0][have]) <= F32 * np.abs(ref[0][have]) + 2.0 ** -16)
    return got


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N,B,V,M", [(1, 1, 1, 1), (1, 1, 1, 4), (2, 3, 5, 7), (1, 4, 1000, 4), (3, 4, 2049, 8),
                                     (2, 8, 50257, 8), (1, 32, 4099, 64), (5, 1, 32000, 1), (2, 2, 131072, 16),
                                     (64, 4, 999, 4), (1, 6, 200003, 12)])
def test_sizes_and_types(dtype, N, B, V, M):
    check(*make(N, B, V, dtype=dtype, seed=V), M)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("fill", [0.0, -3.0, 1e30, "lowest"])
def test_constant_logits_tie_to_the_lowest_index(dtype, fill):
    value = torch.finfo(dtype).min if fill == "lowest" else fill
    x = torch.full((2, 3, 5000), value, dtype=dtype, device="cuda")
    s = torch.tensor([[-1.0, -1.0, -1.0], [-3.0, -1.0, -2.0]], device="cuda")
    got = check(x, s, 8)
    assert got[1][0].tolist() == [0] * 8 and got[2][0].tolist() == list(range(8))
    assert got[1][1].tolist() == [1] * 8


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_few_distinct_values_and_signed_zeros(dtype):
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-1, 2, (3, 4, 30011), generator=g).to(dtype).cuda()
    s = torch.zeros(3, 4, device="cuda")  # beams differ by their log-sums alone
    check(x, s, 33)
    x = torch.zeros(1, 2, 9000, dtype=dtype, device="cuda")
    x[0, :, ::2] = -0.0
    got = check(x, torch.zeros(1, 2, device="cuda"), 6)
    assert got[2][0].tolist() == list(range(6))


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_identical_beams_tie_to_the_first(dtype):
    x, _ = make(1, 1, 4000, dtype=dtype)
    x = x.expand(2, 3, 4000).contiguous()
    got = check(x, torch.full((2, 3), -4.0, device="cuda"), 9)
    assert got[1][:, 0].tolist() == [0, 0]


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_masked_logits(dtype):
    x, s = make(4, 3, 7000, dtype=dtype)
    x[0, 0] = float("-inf")                      # a beam with no continuation
    x[1] = float("-inf")                         # a request with none
    x[2, :, 100:] = float("-inf")                # few left
    x[2, 1, 5] = 3.0
    x[3, 0, :] = torch.finfo(dtype).min          # masked with the lowest value: all equal
    x[3, 1, 1:] = float("-inf")                  # exactly one
    got = check(x, s, 8)
    assert got[1][1].tolist() == [-1] * 8


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_beam_with_nan_or_infinity_is_dead(dtype, bad):
    x, s = make(2, 3, 6000, dtype=dtype)
    x[0, 1, 4321] = bad
    x[1, :, 17] = bad
    got = check(x, s, 6)
    assert 1 not in got[1][0].tolist() and got[1][1].tolist() == [-1] * 6


def test_dead_and_finished_beams():
    x, s = make(5, 4, 3000)
    s[0, 1:] = float("-inf")                     # the first step: one live beam
    s[1, 2] = float("nan")
    s[2, 0] = float("inf")
    x[3, 1] = float("nan")                       # a finished beam's logits are not looked at
    finished = [[0, 0, 0, 0], [0, 1, 0, 0], [0, 0, 0, 1], [1, 1, 1, 1], [1, 0, 1, 0]]
    s[4] = torch.tensor([-0.5, -3.0, -0.5, -2.0])
    got = check(x, s, 6, finished=finished, eos=2999)
    assert got[2][3].tolist() == [2999] * 4 + [-1] * 2
    assert got[1][4].tolist()[:2] == [0, 2]      # equal finished scores: the lower beam first
    check(x, torch.full((5, 4), float("-inf"), device="cuda"), 6, finished=finished, eos=7)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("start", [0, 1, 2, 3, 5, 7])
def test_rows_that_start_anywhere(dtype, start):
    g = torch.Generator().manual_seed(start)
    flat = torch.full((3 * 2 * 2600 + 64,), float("inf"), dtype=dtype, device="cuda")  # read outside a row, it would show
    x = torch.as_strided(flat, (2, 3, 2501), (3 * 2600, 2600 - 3, 1), start + 1)
    x.copy_(torch.randn(2, 3, 2501, generator=g).to(dtype).cuda())
    s = torch.randn(2, 3, generator=g).cuda()
    check(x, s, 10)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_denormal_steps_do_not_lose_candidates(dtype):
    # differences that float64 sums cannot show: any order of the equals is sound, none may be lost or repeated
    x = torch.full((1, 1, 3000), -5.0, dtype=dtype, device="cuda")
    x[0, 0, 10:16] = torch.tensor([0.0, 1e-30, 0.0, 2e-30, -1e-30, 0.0], device="cuda").to(dtype)
    got = binding.kda_beam_select(x, torch.zeros(1, 1, device="cuda"), 6)
    torch.cuda.synchronize()
    assert sorted(got[2][0].tolist()) == list(range(10, 16))


def test_out_workspace_streams_and_graphs():
    x, s = make(3, 4, 40000)
    want = check(x, s, 8)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    floats = binding.kda_beam_select_workspace(3, 4, 40000, 8, BF16, sms)
    work = torch.full((floats + 8,), float("nan"), device="cuda")
    out = tuple(torch.empty_like(t) for t in want)
    got = binding.kda_beam_select(x, s, 8, out=out, workspace=work)
    torch.cuda.synchronize()
    assert all(a is b for a, b in zip(got, out)) and all(torch.equal(a, b) for a, b in zip(want, out))
    assert torch.isnan(work[floats:]).all()
    with pytest.raises(binding.KdaError, match="workspace"):
        binding.kda_beam_select(x, s, 8, workspace=work[:floats - 1])
    side = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for stream in side:
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            results.append(binding.kda_beam_select(x, s, 8))
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(want, r))
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(binding.kda_beam_select(x, s, 8))
        graphs.append(graph)
    x.copy_(make(3, 4, 40000, seed=9)[0])
    want = check(x, s, 8)
    for graph in graphs + graphs:
        graph.replay()
    torch.cuda.synchronize()
    for r in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, r))


def test_empty_batch():
    x, s = make(2, 3, 10)
    got = binding.kda_beam_select(x[:0], s[:0], 4)
    assert [tuple(t.shape) for t in got] == [(0, 4)] * 3


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [3000, 70000, 200001])
@pytest.mark.parametrize("allowed", [1, 5, 40, 3000])
def test_constrained_vocabularies_masked_by_a_finite_value(dtype, V, allowed):
    # all but a few tokens at one low value: far more ties than any list holds
    x, s = make(2, 3, V, dtype=dtype, seed=allowed)
    g = torch.Generator().manual_seed(V)
    keep = torch.zeros(V, dtype=torch.bool)
    keep[torch.randperm(V, generator=g)[:min(allowed, V)]] = True
    x = torch.where(keep.cuda(), x, torch.tensor(-1e9, device="cuda").to(dtype))
    check(x, s, 16)
    check(x, torch.where(torch.arange(3, device="cuda") == 1, s, s - 1e10), 33)  # one beam's masked tokens outrank others'


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_two_values_in_blocks(dtype):
    # the larger value fills whole stretches, so that some groups of threads hold only the smaller one
    x = torch.zeros(1, 2, 90000, dtype=dtype, device="cuda")
    x[0, 0].view(-1, 8)[::32] = 1.0
    x[0, 1, 40000:60000] = 2.0
    check(x, torch.zeros(1, 2, device="cuda"), 64)
    check(x, torch.tensor([[0.0, -5.0]], device="cuda"), 8)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("N,B,V,M", [(1, 16, 150000, 32), (2, 32, 30011, 64), (3, 1, 140000, 64), (40, 16, 999, 32),
                                     (1, 1, 500, 1), (64, 2, 5000, 4)])
def test_many_candidates_and_short_vocabularies(dtype, N, B, V, M):
    check(*make(N, B, V, dtype=dtype, seed=M), M)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_sorted_logits(dtype):
    x = torch.linspace(-9, 9, 100003).expand(2, 2, -1).to(dtype).contiguous().cuda()
    x[1] = x[1].flip(-1)
    check(x, torch.tensor([[0.0, -0.1], [-0.3, 0.0]], device="cuda"), 20)


@pytest.mark.parametrize("num_out", [-1, 0, 65, 2 ** 31 - 1])
def test_a_count_out_of_range_is_refused_before_it_is_allocated(num_out):
    x, s = make(1, 2, 100)
    work = torch.empty(1 << 16, device="cuda")
    for w in (None, work):
        with pytest.raises(binding.KdaError, match="candidates"):
            binding.kda_beam_select(x, s, num_out, workspace=w)

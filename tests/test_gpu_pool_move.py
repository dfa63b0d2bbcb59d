"""GPU tests of kda_pool_move: bit-exact against copies on the host, for forks,
compaction, clearing and in-place permutations, over several pools, element
types, layouts and alignments."""

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from oracle import cache_oracle as co

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def bits(t):
    """The tensor's bits as an integer numpy array (NaN payloads included)."""
    return t.detach().cpu().contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).numpy().copy()


def i32(rows):
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


def check(pools, src, dst, parents=None):
    ref = co.pool_move([bits(p) for p in pools], np.array(src), np.array(dst), None if parents is None else np.array(parents))
    binding.kda_pool_move(pools, i32(src), i32(dst), None if parents is None else i32(parents))
    torch.cuda.synchronize()
    for p, r in zip(pools, ref):
        assert np.array_equal(bits(p), r)


def random_pool(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, dtype=torch.int32).to(torch.int16 if dtype == BF16 else torch.int32) \
        .cuda().view(dtype)


@pytest.mark.parametrize("K", [1, 2, 3, 4, 7, 8, 13, 16, 31, 32])
@pytest.mark.parametrize("shape,dtype", [((2, 128, 128), torch.float32), ((4620,), BF16), ((1,), BF16), ((5, 3), torch.int32)])
def test_random_reorders_in_place(K, shape, dtype):
    rng = np.random.default_rng(K)
    N = 5
    slots = N * K + 3
    own = rng.permutation(np.arange(1, slots))[:N * K].reshape(N, K)
    parents = rng.integers(-1, K + 1, size=(N, K))  # -1 and K are no parents
    parents[0] = np.roll(np.arange(K), 1)           # a full cycle
    parents[1] = np.arange(K)                       # nothing moves
    parents[2] = K - 1                              # one beam takes all
    check([random_pool(slots, *shape, dtype=dtype, seed=K)], own, own, parents)


def test_forks_compaction_and_clearing():
    pool = random_pool(40, 3, 700, dtype=BF16)
    check([pool], [[5], [5], [5], [9]], [[6], [7], [8], [10]])        # forks
    check([pool], [[39], [38], [37]], [[1], [2], [3]])                # compaction
    check([pool], [[0], [-1], [40]], [[11], [12], [13]])              # cleared
    check([pool], [[14], [15], [16], [17]], [[0], [-3], [40], [17]])  # nothing written
    check([pool], [[1, 2]], [[2, 1]])                                 # a swap without parents
    assert torch.count_nonzero(pool.view(torch.int16)[11:14]) == 0


def test_state_conv_and_page_pools_of_several_layers():
    H, slots = 3, 9
    pools = []
    for layer in range(3):
        pools.append(random_pool(slots, H, 128, 128, seed=layer))
        pools.append(random_pool(slots, 3, 3 * H * 128, dtype=BF16, seed=9 + layer).permute(0, 2, 1))  # conv cache strides
    kv = random_pool(slots, 2, 16, H, 64, dtype=BF16, seed=30)
    pools += [kv[:, 0], kv[:, 1]]                                       # interleaved in one allocation
    pools.append(random_pool(slots, H, 16, 64, seed=31).transpose(1, 2))  # head-major pages
    check(pools, [[1, 2, 3], [4, 5, 6]], [[1, 2, 3], [4, 5, 6]], [[2, 0, 0], [1, 1, 2]])


def test_more_pools_than_one_launch_takes():
    pools = [random_pool(6, 10 + i, dtype=BF16 if i % 2 else torch.float32, seed=i) for i in range(130)]
    check(pools, [[1, 2, 3, 4]], [[1, 2, 3, 4]], [[3, 3, 0, 1]])


@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("size", [1, 2, 7, 8, 24, 4097])
def test_alignments_and_odd_sizes(offset, size):
    flat = random_pool(12 * (size + 3) + offset, dtype=BF16)
    pool = torch.as_strided(flat, (12, size), (size + 3, 1), offset)
    check([pool], [[1, 2], [7, 8]], [[2, 1], [9, 10]])
    dense = random_pool(12 * size + 8, dtype=BF16)[:12 * size].view(12, size)
    check([dense], [[3, 4]], [[3, 4]], [[1, 0]])


def test_gaps_between_slots_keep_their_bits():
    flat = random_pool(10, 64)
    before = bits(flat)
    pool = flat[:, :40]
    check([pool], [[1], [2]], [[3], [4]])
    assert np.array_equal(bits(flat)[:, 40:], before[:, 40:])


def test_strided_indices_and_empty_calls():
    pool = random_pool(20, 33)
    ref = co.pool_move([bits(pool)], np.array([[1, 2], [3, 4]]), np.array([[5, 6], [7, 8]]))
    table = i32([[1, 2, 99], [3, 4, 99]])
    binding.kda_pool_move([pool], table[:, :2], i32([[5, 6], [7, 8]]))
    torch.cuda.synchronize()
    assert np.array_equal(bits(pool), ref[0])
    empty = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    binding.kda_pool_move([pool], empty, empty)
    none = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    binding.kda_pool_move([pool], none, none)
    binding.kda_pool_move([pool[:, :0]], i32([[1]]), i32([[2]]))
    torch.cuda.synchronize()
    assert np.array_equal(bits(pool), ref[0])


def test_pool_past_4_gib():
    pool = torch.zeros(40, 1 << 26, dtype=BF16, device="cuda")  # 5 GB, slots of 128 MB
    pool[38, -1], pool[39, -5] = 3.0, 5.0
    binding.kda_pool_move([pool], i32([[38, 39]]), i32([[39, 38]]))
    torch.cuda.synchronize()
    assert float(pool[39, -1]) == 3.0 and float(pool[38, -5]) == 5.0
    assert float(pool[38, -1]) == 0.0 and float(pool[39, -5]) == 0.0


def test_side_stream_and_graph_replay():
    pool = random_pool(9, 5000)
    src, par = i32([[1, 2, 3, 4]]), i32([[1, 2, 3, 0]])
    ref = bits(pool)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.kda_pool_move([pool], src, src, par)
    side.synchronize()
    ref = co.pool_move([ref], src.cpu().numpy(), src.cpu().numpy(), par.cpu().numpy())[0]
    assert np.array_equal(bits(pool), ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.kda_pool_move([pool], src, src, par)
    for parents in ([[1, 2, 3, 0]], [[0, 0, -1, 2]]):
        par.copy_(i32(parents))
        graph.replay()
        torch.cuda.synchronize()
        ref = co.pool_move([ref], src.cpu().numpy(), src.cpu().numpy(), np.array(parents))[0]
        assert np.array_equal(bits(pool), ref)

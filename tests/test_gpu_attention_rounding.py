"""How kda_paged_attention_decode rounds: errors of its arithmetic by their mean and root mean square, beside the
largest ones that the parity tests hold."""

import numpy as np
import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from tests.attention_error import assert_rms, softmax_moments
from tests.rounding import F32, to_np

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


@pytest.mark.parametrize("Hq", [2, 8, 12])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_float32_scores_lean_to_no_side(Hq, sign):
    # One position a sequence and queries of one 1: the log-sum is the key's first channel.
    N = 4096
    g = torch.Generator().manual_seed(Hq)
    key = sign * (1.0 + torch.rand(N, generator=g))
    q = torch.zeros(N, Hq, 64, device="cuda")
    q[:, :, 0] = 1.0
    pages = torch.zeros(N + 1, 16, 1, 64, device="cuda")
    pages[1:, 0, 0, 0] = key.cuda()
    table = torch.arange(1, N + 1, dtype=torch.int32, device="cuda")[:, None]
    _, lse = binding.kda_paged_attention_decode(q, pages, torch.zeros_like(pages), table,
                                                torch.ones(N, dtype=torch.int32, device="cuda"), scale=1.0,
                                                return_lse=True)
    torch.cuda.synchronize()
    off = to_np(lse) / to_np(key)[:, None] - 1.0
    # The score times log2(e) and back by ln 2: the product of the float32 constants is off by `units`; each product
    # rounds by 2^-24 at most, and a key held in two parts is off by 2^-23 at most, to either side alike.  Root mean
    # squares 2^-24 (the parts) and 2^-24 / sqrt(3) twice, over 4096 independent keys: the mean is within
    # 5 * sqrt(5/3) 2^-24 / 64 < 2^-27.
    units = float(np.float32(np.log2(np.e))) * float(np.float32(np.log(2.0))) - 1.0
    assert np.abs(off - units).max() <= 4.01 * F32
    assert np.abs(off.mean(axis=0) - units).max() <= 2.0 ** -27


@pytest.mark.parametrize("Hq", [2, 8, 12])
def test_float32_keys_near_the_largest_float(Hq):
    # a key that rounds past the largest float in fewer bits still has the score of its own
    top = np.array([0x7f7fffff, 0x7f7ff000, 0x7f7fefff, 0x7f7fe000], dtype=np.uint32).view(np.float32)
    key = torch.from_numpy(np.concatenate([top, -top])).repeat(512)
    N = len(key)
    q = torch.zeros(N, Hq, 64, device="cuda")
    q[:, :, 0] = 2.0 ** -126
    pages = torch.zeros(N + 1, 16, 1, 64, device="cuda")
    pages[1:, 0, 0, 0] = key.cuda()
    table = torch.arange(1, N + 1, dtype=torch.int32, device="cuda")[:, None]
    _, lse = binding.kda_paged_attention_decode(q, pages, torch.zeros_like(pages), table,
                                                torch.ones(N, dtype=torch.int32, device="cuda"), scale=1.0,
                                                return_lse=True)
    torch.cuda.synchronize()
    # exact product (a power of two), the two constants and products of the test above: 4 half steps bound them
    assert np.abs(to_np(lse) / (to_np(key)[:, None] * 2.0 ** -126) - 1.0).max() <= 4.01 * F32


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 32, 8), (128, 32, 8), (256, 16, 4), (64, 24, 2), (128, 24, 2), (256, 24, 2)])
@pytest.mark.parametrize("length,window", [(1000, 0), (70001, 0), (70001, 5000)])
def test_outputs_are_off_by_their_rounding_alone(dtype, D, Hq, Hkv, length, window):
    # six sequences that share their pages, of slightly different lengths
    N, page = 6, 64
    P = -(-length // page)
    g = torch.Generator(device="cuda").manual_seed(D + Hq + length)
    k, v = (torch.randn(P + 1, page, Hkv, D, device="cuda", generator=g).to(dtype) for _ in range(2))
    q = torch.randn(N, Hq, D, device="cuda", generator=g).to(dtype)
    table = (torch.randperm(P, device="cuda", generator=g) + 1).to(torch.int32).expand(N, P).contiguous()
    lens = [length - 13 * n for n in range(N)]
    out, lse = binding.kda_paged_attention_decode(q, k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                                  window=window, return_lse=True)
    keys, values = (to_np(x[table[0].long()].flatten(0, 1).transpose(0, 1)) for x in (k, v))
    G, scale = Hq // Hkv, D ** -0.5
    queries = to_np(q)
    ref, ref_lse = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    weighted, spread = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    for h in range(Hkv):
        for n in range(N):
            first = max(0, lens[n] - window) if window else 0
            heads = slice(h * G, (h + 1) * G)
            ref[n, heads], ref_lse[n, heads], weighted[n, heads], spread[n, heads] = softmax_moments(
                queries[n, heads], keys[h, first:lens[n]], values[h, first:lens[n]], scale)
    # 64 roundings in a score's product; weights in two bfloat16 (2^-16), or in float32's two parts (2^-20)
    score = 64 * F32 * np.linalg.norm(queries, axis=-1).max() * np.linalg.norm(keys, axis=-1).max() * scale
    assert_rms(to_np(out), ref, weighted, spread, score, 2.0 ** -16 if dtype is BF16 else 2.0 ** -20, "out")
    # a log-sum: the scores' errors average, 2^-22 of the exponential, 512 roundings of its sums, its own 2^-24
    assert np.abs(to_np(lse) - ref_lse).max() <= score + 2.0 ** -22 + 512 * F32 + F32 * np.abs(ref_lse).max()

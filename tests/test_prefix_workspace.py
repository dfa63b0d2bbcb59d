"""The workspace of kda_prefix_attention_decode (CPU only): no more than the paged call's where no call shares."""

import pytest
import torch

from linear_attention_decode_02_gb300 import binding
from tests.test_cache_abi import BF16, lib  # noqa: F401

FP32 = torch.float32


@pytest.mark.parametrize("sequences", [1, 512, 4096])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 256), (4, 4, 256), (5, 1, 64), (32, 2, 128), (64, 8, 64)])
def test_float32_heads_that_never_share_need_the_paged_workspace(lib, sequences, Hq, Hkv, D):  # noqa: F811
    alone = binding.kda_paged_attention_workspace(Hq, Hkv, D, FP32, 152)
    assert binding.kda_prefix_attention_workspace(sequences, Hq, Hkv, D, FP32, 152) == alone
    assert binding.kda_prefix_attention_workspace(sequences, Hq, Hkv, D, BF16, 152) > \
        binding.kda_paged_attention_workspace(Hq, Hkv, D, BF16, 152)


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (4, 1, 64), (16, 16, 64)])
def test_float32_heads_that_may_share_need_parts_of_every_sequence(lib, Hq, Hkv, D):  # noqa: F811
    few, many = (binding.kda_prefix_attention_workspace(n, Hq, Hkv, D, FP32, 152) for n in (512, 4096))
    assert many - few >= 3584 * 2 * 8 * Hq * D  # outputs of eight warps, of common and of own positions

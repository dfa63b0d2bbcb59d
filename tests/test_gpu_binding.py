"""What the Python binding of the cache and beam calls refuses by itself, and what it keeps."""

import gc

import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


def outputs(N, M):
    return (torch.zeros(N, M, device="cuda"), *(torch.zeros(N, M, dtype=torch.int32, device="cuda") for _ in range(2)))


@pytest.mark.parametrize("columns", [3, 5, 64])
def test_beam_outputs_of_another_count_are_refused(columns):
    # whatever was called before: a larger call leaves a larger workspace
    x, s = torch.randn(2, 4, 5000, device="cuda"), torch.zeros(2, 4, device="cuda")
    for before in (4, 64):
        binding.kda_beam_select(x, s, before)
        out = outputs(2, columns)
        with pytest.raises(ValueError, match="num_out is 4"):
            binding.kda_beam_select(x, s, 4, out=out)
        assert all(torch.count_nonzero(t) == 0 for t in out)
    with pytest.raises(ValueError, match="num_out is 4"):
        binding.kda_beam_select(x, s, 4, out=tuple(t.flatten() for t in outputs(2, 4)))
    got = binding.kda_beam_select(x, s, 4, out=outputs(2, 4))
    assert all(torch.equal(a, b) for a, b in zip(got, binding.kda_beam_select(x, s, 4)))


def test_large_workspaces_are_not_kept():
    x = torch.randn(1024, 32, 512, device="cuda").to(BF16)
    s = torch.zeros(1024, 32, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert binding.kda_beam_select_workspace(1024, 32, 512, 64, BF16, sms) > 4 << 20
    assert binding.kda_paged_attention_workspace(4096, 1, 256, BF16, sms) <= 4 << 20
    small = binding.kda_beam_select(x[:2], s[:2], 64)
    torch.cuda.synchronize()
    gc.collect()  # nothing of another test's goes meanwhile
    before = torch.cuda.memory_allocated()
    first = binding.kda_beam_select(x, s, 64)
    again = binding.kda_beam_select(x, s, 64)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert all(torch.equal(a[:2], b) for a, b in zip(first, small))
    results = sum(-(-t.numel() * t.element_size() // 512) * 512 for t in first + again)
    assert torch.cuda.memory_allocated() - before == results

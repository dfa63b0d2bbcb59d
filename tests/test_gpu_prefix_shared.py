"""More of kda_prefix_attention_decode on the GPU: calls whose sequences do share, by the rule, with what the first tests
leave out."""

import pytest
import torch

from linear_attention_decode_02_gb300 import binding, build
from tests.test_gpu_paged_attention import same
from tests.test_gpu_prefix_attention import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


@pytest.mark.parametrize("page", [64, 24])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_units_of_an_odd_number_of_tiles(D, page):
    """Behind a unit of an odd number of tiles the two lanes change places in the ring of keys and values."""
    groups = [(128 * tiles - e, [3, 40]) for tiles in (3, 2, 5, 1, 2, 7, 3, 4) for e in (0, 1, 65)] * 4
    c = make(groups, Hq=16, Hkv=16, D=D, page=page)
    out, lse = check(c)
    for _ in range(20):
        again, sums = run(c)
        assert same(again, out) and same(sums, lse)
    torch.cuda.synchronize()
    assert binding.kda_device_error() == 0

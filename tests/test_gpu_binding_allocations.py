"""What the binding's calls allocate goes through PyTorch's dispatcher: modes and deterministic fills see it."""

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.utils._python_dispatch import TorchDispatchMode

from linear_attention_decode_02_gb300 import binding, build

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.library()


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        if func.overloadpacket is torch.ops.aten.empty:
            self.shapes.append(tuple(args[0]))
        return func(*args, **(kwargs or {}))


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32, device="cuda")


def cache():
    return torch.zeros(4, 8, 2, 64, dtype=BF16, device="cuda"), torch.zeros(4, 8, 2, 64, dtype=BF16, device="cuda")


def rope(axes):
    q, k, v = (torch.zeros(3, h, 64, dtype=BF16, device="cuda") for h in (4, 2, 2))
    steps = binding.kda_rope_phase_steps(64)
    if axes:
        return lambda: binding.kda_rope_axes_append(q, k, v, steps, i32(32), i32(3, 2), i32(3), *cache())
    return lambda: binding.kda_rope_append(q, k, v, steps, i32(3), i32(3, 2), *cache())


def attention(shared):
    q = torch.zeros(3, 4, 64, dtype=BF16, device="cuda")
    more = (i32(2), i32(1)) if shared else ()
    call = binding.kda_prefix_attention_decode if shared else binding.kda_paged_attention_decode
    args = (q, *cache(), i32(3, 2), i32(3), *more)
    return lambda: call(*args, return_lse=True)


CALLS = {"rope": (lambda: rope(False), [(3, 4, 64)]), "rope axes": (lambda: rope(True), [(3, 4, 64)]),
         "attention": (lambda: attention(False), [(3, 4, 64), (3, 4)]),
         "shared attention": (lambda: attention(True), [(3, 4, 64), (3, 4)]),
         "beams": (lambda: lambda: binding.kda_beam_select(torch.zeros(2, 4, 500, device="cuda"), torch.zeros(2, 4, device="cuda"), 3),
                   [(2, 3)] * 3),
         "pages": (lambda: lambda: binding.kda_page_assign(i32(3), i32(3), i32(3, 2), i32(9), i32(2), 8, 5),
                   [(3,), (2,), (4,), (5,)])}


@pytest.mark.parametrize("name", CALLS)
def test_a_dispatch_mode_sees_the_outputs_allocated(name):
    make, shapes = CALLS[name]
    call = make()
    with Seen() as seen:
        call()
    torch.cuda.synchronize()
    found = list(seen.shapes)
    for shape in shapes:
        assert shape in found, (shape, seen.shapes)
        found.remove(shape)


def test_a_profiler_sees_the_outputs_allocated():
    call = CALLS["pages"][0]()
    call()
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as seen:
        for _ in range(3):
            i32(1), call()
    torch.cuda.synchronize()
    counts = {e.key: e.count for e in seen.key_averages()}
    assert counts.get("aten::empty", 0) >= 3 * 4 + counts.get("aten::zeros", 0), counts


def test_calls_under_inference_mode_and_deterministic_fills():
    lens, table, ring, state = i32(3), i32(3, 2), torch.arange(1, 10, dtype=torch.int32, device="cuda"), i32(2)
    state[1] = 9

    def call():
        return binding.kda_page_assign(lens, lens + 5, table.clone(), ring.clone(), state, 8, 15)

    wanted = call()
    with torch.inference_mode():
        got = call()
    assert all(t.is_inference() for t in got) and all(torch.equal(a, b) for a, b in zip(got, wanted))
    torch.use_deterministic_algorithms(True)
    try:
        got = call()
    finally:
        torch.use_deterministic_algorithms(False)
    assert all(torch.equal(a, b) for a, b in zip(got, wanted))


@pytest.mark.parametrize("name", ["attention", "beams"])
def test_a_workspace_is_not_kept_from_a_mode_that_gives_no_memory(name):
    x, s = torch.randn(2, 4, 500, device="cuda"), torch.zeros(2, 4, device="cuda")
    call = attention(False) if name == "attention" else lambda: binding.kda_beam_select(x, s, 3)
    wanted = call()
    stream = torch.cuda.Stream()  # without a workspace of its own yet
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        with FakeTensorMode():
            with pytest.raises(Exception):
                call()
        got = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, wanted))

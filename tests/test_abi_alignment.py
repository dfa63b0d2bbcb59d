"""Every tensor of every entry point has to start on a boundary of its elements (CPU only: descriptors moved on by a
byte or two, which no torch tensor is but a C caller's packed buffer may be; refused before any launch)."""

import pytest
import torch

from linear_attention_decode_02_gb300.binding import desc
from tests import test_abi as recurrent
from tests import test_cache_abi as cache
from tests.test_cache_abi import INVALID, lib  # noqa: F401

CALLS = {
    "recurrent": (recurrent._recurrent_args, recurrent._call_recurrent),
    "packed": (recurrent._packed_args, recurrent._call_packed),
    "fused": (recurrent._fused_args, recurrent._call_fused),
    "spec": (recurrent._spec_args, recurrent._call_spec),
    "packed fused": (recurrent._pf_args, recurrent._call_pf),
    "rope": (lambda: {**cache._rope(), "cu": torch.zeros(4, dtype=torch.int32)}, cache._call_rope),
    "attention": (cache._attend, cache._call_attend),
    "attention f32": (lambda: cache._attend(dtype=torch.float32), cache._call_attend),
    "beam": (cache._beam, cache._call_beam),
    "move": (lambda: dict(pool=torch.zeros(5, 6, dtype=torch.bfloat16), other=torch.zeros(5, 4), src=cache._i32(2, 3),
                          dst=cache._i32(2, 3), parents=cache._i32(2, 3)),
             lambda lib, t: cache._move(lib, [t["pool"], t["other"]], t["src"], t["dst"], t["parents"])),
}


@pytest.mark.parametrize("op,name", [(op, name) for op, (make, _) in CALLS.items() if "attention" not in op and op != "beam"
                                     for name in make()] +
                         [(op, name) for op in ("attention", "attention f32")
                          for name in ("q", "k_pages", "v_pages", "table", "lens", "work", "out", "lse")] +
                         [("beam", name) for name in ("logits", "scores", "finished", "work", "s", "p", "t")])
def test_tensors_off_their_elements_boundaries_are_refused(lib, monkeypatch, op, name):
    make, call = CALLS[op]
    t = make()
    for by in range(1, t[name].element_size()):
        def moved(x):
            d = desc(x)
            if x is t[name]:
                d.data += by
            return d
        monkeypatch.setattr(recurrent, "desc", moved)
        monkeypatch.setattr(cache, "desc", moved)
        # the recurrent call takes ready descriptors as they are
        given = {**t, name: moved(t[name])} if op == "recurrent" else t
        assert call(lib, given) == INVALID, (by, lib.kda_last_error_message())
        assert "aligned" in lib.kda_last_error_message().decode()

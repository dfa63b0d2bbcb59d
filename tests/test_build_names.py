"""The CPython module is compiled to one interpreter's and one PyTorch's binary interface, and carries both in its name
(CPU only)."""

import os
import platform
import sys

import torch

from linear_attention_decode_02_gb300 import binding, build


def test_module_is_named_for_what_it_was_built_for():
    assert build.PYLIB == binding.module_path(torch.__version__) == binding._MODULE_PATH
    name = os.path.basename(build.PYLIB)
    for part in (sys.implementation.cache_tag, platform.machine(), torch.__version__):
        assert part in name
    build.build()
    assert build.up_to_date() and binding._native().__file__ == build.PYLIB


def test_a_module_of_another_torch_is_neither_up_to_date_nor_loaded(monkeypatch):
    build.build()
    other = binding.module_path("0.0.0")
    assert other != build.PYLIB
    monkeypatch.setattr(build, "PYLIB", other)
    assert not build.up_to_date()
    monkeypatch.setattr(binding, "_MODULE_PATH", other)
    monkeypatch.setattr(binding, "_module", None)
    try:
        binding._native()
    except RuntimeError as e:
        assert "not built" in str(e)
    else:
        raise AssertionError("loaded a module that does not exist")

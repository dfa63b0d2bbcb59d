"""Page assignment, rotary positions with several axes and shared-prefix attention from C:
`tests/c_client/kda_pages_c_client.c` compiled as strict C99 against include/kda.h, linked and run (no GPU needed)."""

import os
import shutil
import subprocess

import pytest

from linear_attention_decode_02_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_pages_c_client_compiles_links_and_runs(tmp_path):
    build.build()
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    lib_dir = os.path.join(ROOT, "linear_attention_decode_02_gb300")
    exe = tmp_path / "kda_pages_c_client"
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c_client", "kda_pages_c_client.c"), "-L", lib_dir, "-lkda",
                    "-Wl,-rpath," + lib_dir, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert "all checks passed" in r.stdout

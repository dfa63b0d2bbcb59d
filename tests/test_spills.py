"""Registers of the float32 tensor-core attention kernels, by the compiler's own report (CPU only): all is held in
registers, also where they have every one."""

import os
import re
import subprocess

from linear_attention_decode_02_gb300 import build


def test_float32_attention_spills_nothing(tmp_path):
    log = subprocess.run([build._nvcc(), *build.NVCC_FLAGS, *build.ARCH, "-Xptxas=-v", "-c",
                          os.path.join(build.CSRC, "kda_attend_tf32.cu"), "-o", str(tmp_path / "x.o")],
                         capture_output=True, text=True, check=True).stderr
    found = re.findall(r"Function properties for (\S+)\n\s*(\d+) bytes stack frame, (\d+) bytes spill stores", log)
    assert len(found) == 12, log
    assert [(name, s) for name, _, s in found if s != "0"] == []

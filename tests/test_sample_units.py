"""The row sampler's constants on the host (no GPU): top_search_resident_amd/csrc/
sample_units.hpp, the header the library uses, gives the nearest whole numbers,
also on a thread that flushes subnormals to zero (torch.set_flush_denormal)."""
import os
import platform
import shutil
import subprocess

import pytest

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "sanitize")


@pytest.mark.skipif(shutil.which("g++") is None or platform.machine() != "x86_64", reason="no host x86 C++ compiler")
@pytest.mark.parametrize("flags", [["-O2"], ["-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all"]])
def test_units_with_and_without_subnormals(tmp_path, flags):
    exe = str(tmp_path / "units_driver")
    for cmd in (["g++", "-std=c++17", *flags, "-o", exe, os.path.join(HERE, "units_driver.cpp")], [exe]):
        res = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
        assert res.returncode == 0, " ".join(cmd) + "\n" + res.stdout + res.stderr
    assert res.stdout.strip() == "ok"

"""The workspace of the MoE layer for a few tokens, replayed on the host by
tests/moe_few_layout_driver.cpp with the arithmetic that the kernels use
(csrc/moe_few_layout.hpp): every write and load stays inside the smallest
workspace a call may have, for every number of tokens of an expert. CPU only;
skipped without g++."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_write_and_load_of_the_workspace(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "moe_few_layout")
    build = subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-o", exe,
                            os.path.join(ROOT, "tests", "moe_few_layout_driver.cpp")], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr[-4000:]
    assert "in place" in run.stdout

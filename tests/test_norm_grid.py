"""The launch geometry of the norm's gradient in any layout on the host
(tests/norm_grid_driver.cpp). CPU only; skipped without g++ or the HIP headers."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIP_INCLUDE = "/opt/rocm/include"


def test_columns_up_to_the_limit_fit_the_grid(tmp_path):
    if shutil.which("g++") is None or not os.path.isdir(HIP_INCLUDE):
        pytest.skip("no g++ or no HIP headers")
    exe = str(tmp_path / "norm_grid")
    build = subprocess.run(["g++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I" + HIP_INCLUDE, "-o", exe,
                            os.path.join(ROOT, "tests", "norm_grid_driver.cpp")], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stderr[-4000:]

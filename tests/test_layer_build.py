"""The layer's device code compiles without a warning (an access type whose
alignment the compiler does not lower is one, and its static assertions hold).
CPU only; skipped without hipcc."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_scaled_gemm_amax_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"


@pytest.mark.parametrize("source", ["norm.hip", "swiglu.hip", "moe_few.hip"])
def test_no_warnings(source):
    if not os.path.exists(HIPCC):
        pytest.skip("no hipcc")
    out = subprocess.run([HIPCC, "--offload-arch=gfx950", "-std=c++17", "-ffp-contract=off", "-Wall", "-Werror",
                          "-Wno-unused-command-line-argument", "-Xclang", "-target-feature", "-Xclang",
                          "-packed-fp32-ops", "--cuda-device-only", "-O0", "-c", "-o", os.devnull,
                          os.path.join(CSRC, source)],
                         capture_output=True, text=True)
    assert out.returncode == 0 and "warning" not in out.stderr, out.stderr[-3000:]

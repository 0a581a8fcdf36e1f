"""Refusals of the layer's entry points, on the host before anything is launched:
the C ABI with addresses that are never used, the Python binding with CPU
tensors; and the assembly of their kernels (no scratch memory). CPU only."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_scaled_gemm_amax_amd", "csrc")
A = ctypes.c_void_p(0x10000)
IA, AL, UN = 1, 2, 3


def off(n):
    return ctypes.c_void_p(0x10000 + n)


@pytest.fixture(scope="module")
def fp8():
    import fp8_scaled_gemm_amax_amd as m
    return m


def refuse(fp8, name, good, changes):
    """Every change of the good arguments ({position: value}, status) is refused so,
    with a message that names the function."""
    for change, status in changes:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert getattr(fp8.lib, name)(*args) == status, (change, fp8.lib.fp8_last_error())
        assert name.encode() in fp8.lib.fp8_last_error(), change


def test_norm_quantize_row(fp8):
    #       0  1  2   3   4  5  6  7     8  9  10 11 12  13 14 15  16 17 18 19 20  21 22 23
    good = [A, 4, 64, 64, A, A, 0, 1e-5, 0, 0, 0, A, 64, A, A, 64, A, A, A, 0, 64, A, 4, None]
    refuse(fp8, "fp8_norm_quantize_row", good, [
        ({0: None}, IA), ({1: -1}, IA), ({2: 0, 3: 64}, IA), ({3: 63}, IA), ({6: 2}, IA), ({7: -1.0}, IA),
        ({7: float("nan")}, IA), ({7: float("inf")}, IA), ({8: 2}, IA), ({9: 4}, IA), ({10: 33}, IA),
        ({11: None, 13: None, 14: None}, IA), ({13: None}, IA), ({11: None}, IA), ({12: 63}, IA), ({15: 63}, IA),
        ({18: None}, IA), ({21: None}, IA), ({19: 2}, IA), ({20: 63}, IA), ({22: 3}, IA), ({2: 48, 20: 48}, IA),
        ({0: off(1)}, AL), ({4: off(1)}, AL), ({6: 1, 5: off(2)}, AL), ({13: off(2)}, AL), ({14: off(1)}, AL),
        ({17: off(2)}, AL), ({18: off(4)}, AL), ({20: 68}, AL), ({21: off(2)}, AL), ({0: off(8)}, AL), ({3: 66}, AL),
        ({12: 66}, AL), ({4: off(2)}, AL),
        ({1: 1 << 30, 22: 1 << 30}, UN), ({2: 16416, 3: 16416, 12: 16416, 15: 16416, 20: 16416}, UN)])


def test_norm_backward(fp8):
    #       0  1  2   3   4  5   6  7  8  9  10 11 12  13 14 15 16       17
    good = [A, 4, 64, 64, A, 64, A, 0, A, A, 0, A, 64, A, A, A, 4 * 512, None]
    assert fp8.lib.fp8_norm_backward_workspace(4, 64) == 4 * 2 * 64 * 4 == 4 * 512
    refuse(fp8, "fp8_norm_backward", good, [
        ({0: None}, IA), ({4: None}, IA), ({11: None}, IA), ({9: None}, IA), ({8: None}, IA), ({2: 0}, IA),
        ({3: 60}, IA), ({5: 60}, IA), ({12: 60}, IA), ({7: 3}, IA), ({10: -1}, IA), ({15: None}, IA), ({16: 2047}, IA),
        ({0: off(1)}, AL), ({4: off(1)}, AL), ({11: off(1)}, AL), ({8: off(2)}, AL), ({9: off(1)}, AL),
        ({13: off(2)}, AL), ({14: off(2)}, AL), ({15: off(8)}, AL), ({6: off(1)}, AL), ({1: 1 << 30}, UN),
        ({2: 1 << 27, 3: 1 << 27, 5: 1 << 27, 12: 1 << 27, 16: 1 << 40}, UN)])


def test_norm_workspace_sizes(fp8):
    w = fp8.lib.fp8_norm_backward_workspace
    assert w(1, 1) == 8 and w(100000, 8) == 512 * 2 * 8 * 4
    assert w(0, 8) == w(8, 0) == w(-1, 8) == w(1 << 30, 8) == w(8, 1 << 27) == 0
    assert w(1, (1 << 27) - 1) == 8 * ((1 << 27) - 1)


def test_mx_norm_backward(fp8):
    #       0  1  2   3   4  5  6   7  8  9  10 11 12 13 14 15  16 17 18 19  20 21   22
    good = [A, 4, 64, 64, A, 0, 64, A, 4, A, A, 0, A, 0, A, 64, A, A, A, 64, A, 2048, None]
    refuse(fp8, "fp8_mx_norm_backward", good, [
        ({0: None}, IA), ({4: None}, IA), ({7: None}, IA), ({12: None}, IA), ({5: 2}, IA), ({8: 3}, IA), ({6: 60}, IA),
        ({2: 40, 6: 40}, IA), ({19: 63}, IA), ({20: None}, IA), ({21: 0}, IA), ({11: 5}, IA), ({13: 9}, IA),
        ({4: off(4)}, AL), ({6: 68}, AL), ({7: off(1)}, AL), ({0: off(2)}, AL), ({3: 66}, AL), ({14: off(8)}, AL),
        ({18: off(8)}, AL), ({9: off(2)}, AL), ({10: off(2)}, AL), ({20: off(4)}, AL),
        ({2: 16416, 3: 16416, 6: 16416, 15: 16416, 19: 16416, 21: 1 << 40}, UN), ({1: 1 << 30, 8: 1 << 30}, UN)])


def test_swiglu_quantize_row_mx(fp8):
    #       0  1  2   3    4  5  6  7   8  9  10 11   12 13 14
    good = [A, 4, 64, 128, 0, 0, A, 64, A, A, 0, 128, A, 4, None]
    refuse(fp8, "fp8_swiglu_quantize_row_mx", good, [
        ({0: None}, IA), ({1: -2}, IA), ({2: -32}, IA), ({2: 1 << 30}, IA), ({2: 48}, IA), ({3: 127}, IA), ({4: 9}, IA),
        ({5: -1}, IA), ({6: None}, IA), ({7: 32}, IA), ({8: None}, IA), ({9: None}, IA), ({10: 3}, IA), ({11: 64}, IA),
        ({12: None}, IA), ({13: 3}, IA), ({0: off(8)}, AL), ({3: 132}, AL), ({6: off(4)}, AL), ({7: 68}, AL),
        ({8: off(2)}, AL), ({9: off(4)}, AL), ({11: 132}, AL), ({12: off(1)}, AL), ({1: 1 << 26, 13: 1 << 26}, UN),
        ({2: 16416, 3: 32832, 7: 16416, 11: 32832}, UN)])


def test_swiglu_backward(fp8):
    #       0  1  2   3   4  5    6  7    8  9   10
    good = [A, 4, 40, 40, A, 80, A, 80, A, 40, None]
    refuse(fp8, "fp8_swiglu_backward", good, [
        ({0: None}, IA), ({4: None}, IA), ({6: None}, IA), ({1: -1}, IA), ({2: -8}, IA), ({3: 32}, IA), ({5: 72}, IA),
        ({7: 72}, IA), ({9: 32}, IA), ({2: 36}, AL), ({0: off(8)}, AL), ({3: 44}, AL), ({4: off(8)}, AL), ({5: 84}, AL),
        ({6: off(8)}, AL), ({7: 84}, AL), ({8: off(8)}, AL), ({9: 44}, AL), ({1: 1 << 30}, UN)])
    good = [A, 4, 64, 64, A, 0, 128, A, 4, A, 128, A, 64, None]
    refuse(fp8, "fp8_mx_swiglu_backward", good, [
        ({4: None}, IA), ({7: None}, IA), ({5: 2}, IA), ({6: 120}, IA), ({8: 3}, IA), ({2: 40, 3: 40}, IA),
        ({4: off(4)}, AL), ({6: 132}, AL), ({7: off(2)}, AL), ({9: off(8)}, AL), ({1: 1 << 30, 8: 1 << 30}, UN)])


def test_moe_few_tokens(fp8):
    #       0  1  2    3    4  5  6  7  8  9  10   11          12 13 14 15  16        17 18  19 20   21 22             23
    good = [A, 4, 128, 128, A, A, 2, 8, A, 0, 128, 128 * 128, A, A, 0, 64, 64 * 128, A, 64, A, 128, A, 4 * 2 * 64 * 4,
            None]
    refuse(fp8, "fp8_moe_few_tokens", good, [
        ({0: None}, IA), ({4: None}, IA), ({5: None}, IA), ({8: None}, IA), ({12: None}, IA), ({13: None}, IA),
        ({17: None}, IA), ({19: None}, IA), ({21: None}, IA), ({22: 2047}, IA), ({1: -1}, IA), ({2: 120}, IA),
        ({2: 0}, IA), ({18: 72}, IA), ({18: 0}, IA), ({18: 1 << 20}, IA), ({3: 120}, IA), ({20: 120}, IA), ({6: 0}, IA),
        ({6: 65}, IA), ({7: 0}, IA), ({7: 1025}, IA), ({9: 4}, IA), ({10: 112}, IA), ({15: 48}, IA), ({11: -16}, IA),
        ({16: -16}, IA), ({0: off(8)}, AL), ({3: 132}, AL), ({8: off(8)}, AL), ({10: 136}, AL), ({11: 8}, AL),
        ({13: off(4)}, AL), ({15: 72}, AL), ({16: 24}, AL), ({4: off(2)}, AL), ({5: off(1)}, AL), ({12: off(2)}, AL),
        ({17: off(2)}, AL), ({19: off(1)}, AL), ({21: off(8)}, AL), ({9: 2}, UN), ({14: 3}, UN), ({1: 65, 22: 1 << 20},
                                                                                                 UN)])


# ------------------------------------------------------------------ Python --
def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def f32(*s):
    return torch.zeros(s)


def bad(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_python_norm(fp8):
    n = fp8.fp8_norm_quantize_row
    args = lambda **k: dict(dict(x=bf(4, 64), gamma=bf(64), beta=bf(64), eps=1e-5, kind=0, fmt=0, margin=0,  # noqa: E731
                                 q=u8(4, 64), scale_inv_out=f32(4)), **k)
    bad("on a GPU", n, **args())
    bad("bfloat16", n, **args(x=f32(4, 64)))
    bad("rows overlap", n, **args(x=bf(64).expand(4, 64)))
    bad("unit stride", n, **args(x=bf(64, 4).t()))
    bad("gamma", n, **args(gamma=bf(63)))
    bad("beta", n, **args(beta=f32(64)))
    bad("bfloat16 or float32", n, **args(gamma=torch.zeros(64, dtype=torch.float64), beta=None))
    bad("q must be", n, **args(q=u8(4, 63)))
    bad("scale_inv_out", n, **args(scale_inv_out=f32(5)))
    bad("y must be", n, **args(y=bf(5, 64)))
    bad("rstd_out", n, **args(rstd_out=torch.zeros(4, dtype=torch.float64)))
    bad("scale records", n, **args(xhat_q=u8(4, 64)))
    bad("needs xhat_q", n, **args(xhat_scale=u8(1, 4, 4)))
    bad("scale records must be", n, **args(xhat_q=u8(4, 64), xhat_scale=u8(2, 4, 4)))
    g = fp8.fp8_norm_backward
    back = lambda **k: dict(dict(dy=bf(4, 64), x=bf(4, 64), gamma=None, mean=f32(4), rstd=f32(4), kind=0,  # noqa: E731
                                 dx=bf(4, 64)), **k)
    bad("on a GPU", g, **back())
    bad("rows overlap", g, **back(dy=bf(64).expand(4, 64)))
    bad("dx must be", g, **back(dx=bf(4, 32)))
    bad("mean", g, **back(mean=f32(3)))
    bad("dgamma", g, **back(dgamma=bf(64)))
    bad("workspace must be contiguous", g, **back(workspace=f32(10, 10).t()))
    m = fp8.fp8_mx_norm_backward
    bad("xhat_q must be", m, bf(4, 64), u8(4, 32), 0, u8(1, 4, 4), None, None, f32(4), 0, bf(4, 64))
    bad("scale records", m, bf(4, 64), u8(4, 64), 0, None, None, None, f32(4), 0, bf(4, 64))


def test_python_swiglu(fp8):
    s = fp8.fp8_swiglu_quantize_row_mx
    bad("on a GPU", s, bf(4, 128), 0, 0, u8(4, 64), f32(4), u8(4, 128), 0, u8(1, 4, 4))
    bad("even number", s, bf(4, 127), 0, 0, u8(4, 64), f32(4), u8(4, 128), 0, u8(1, 4, 4))
    bad("q must be", s, bf(4, 128), 0, 0, u8(4, 128), f32(4), u8(4, 128), 0, u8(1, 4, 4))
    bad("hq must be", s, bf(4, 128), 0, 0, u8(4, 64), f32(4), u8(4, 64), 0, u8(1, 4, 4))
    b = fp8.fp8_swiglu_backward
    bad("on a GPU", b, bf(4, 64), bf(4, 128), bf(4, 128))
    bad("h must be", b, bf(4, 64), bf(4, 64), bf(4, 128))
    bad("rows overlap", b, bf(64).expand(4, 64), bf(4, 128), bf(4, 128))
    bad("a must be", b, bf(4, 64), bf(4, 128), bf(4, 128), a=bf(4, 128))
    bad("scale records must be", fp8.fp8_mx_swiglu_backward, bf(4, 64), u8(4, 128), 0, u8(1, 5, 4), bf(4, 128))


def test_python_moe(fp8):
    m = fp8.fp8_moe_few_tokens
    args = lambda **k: dict(dict(  # noqa: E731
        x=bf(3, 64), expert_idx=torch.zeros((3, 2), dtype=torch.int32), weights=f32(3, 2), w1=u8(4, 64, 64), f1=0,
        w1_scale_inv=f32(4, 64), w2=u8(4, 64, 32), f2=0, w2_scale_inv=f32(4, 64), out=bf(3, 64), workspace=f32(6, 32)),
        **k)
    bad("on a GPU", m, **args())
    bad("expert_idx", m, **args(expert_idx=torch.zeros((3, 2), dtype=torch.int64)))
    bad("rows, x has", m, **args(expert_idx=torch.zeros((2, 2), dtype=torch.int32)))
    bad("weights", m, **args(weights=f32(3, 1)))
    bad("do not match", m, **args(w1=u8(4, 64, 32)))
    bad("do not match", m, **args(w2=u8(3, 64, 32)))
    bad("do not overlap", m, **args(w1=u8(4, 1, 64).expand(4, 64, 64)))
    bad("w1_scale_inv", m, **args(w1_scale_inv=f32(4, 32)))
    bad("out must be", m, **args(out=bf(2, 64)))


# ---------------------------------------------------------------- assembly --
@pytest.mark.parametrize("source", ["norm.hip", "swiglu.hip", "moe_few.hip"])
def test_no_scratch(source):
    out = subprocess.run(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", "-O3", "-std=c++17", "-ffp-contract=off",
                          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S", "-o",
                          "-", os.path.join(CSRC, source)], capture_output=True, text=True)
    assert out.returncode == 0, out.stderr[-2000:]
    sizes = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", out.stdout)
    assert sizes and all(int(s) == 0 for s in sizes), "a kernel uses scratch memory"
    assert "scratch_" not in out.stdout

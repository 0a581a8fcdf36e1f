"""Refusals of the block's entry points (the residual's addition with the norm, the
gated products, adapters), on the host before anything is launched: the C ABI with
addresses that are never used, the Python binding with CPU tensors; their kernels
compile without a warning and use no scratch memory. CPU only."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from test_layer_api import refuse

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_scaled_gemm_amax_amd", "csrc")
HIPCC = "/opt/rocm/bin/hipcc"
A = ctypes.c_void_p(0x10000)
IA, AL, UN = 1, 2, 3


def off(n):
    return ctypes.c_void_p(0x10000 + n)


@pytest.fixture(scope="module")
def fp8():
    import fp8_scaled_gemm_amax_amd as m
    return m


def test_add_norm_quantize_row(fp8):
    #       x  r  c   ldx res ld sum ld  g  b  w  eps  k  f  mg q  ldq si y  ldy m  rs xq xf ld  xs ls st
    #       0  1  2   3   4  5   6  7   8  9  10 11   12 13 14 15 16  17 18 19  20 21 22 23 24  25 26 27
    good = [A, 4, 64, 64, A, 64, A, 64, A, A, 0, 1e-5, 0, 0, 0, A, 64, A, A, 64, A, A, A, 0, 64, A, 4, None]
    refuse(fp8, "fp8_add_norm_quantize_row", good, [
        ({0: None}, IA), ({1: -1}, IA), ({2: 0, 3: 64}, IA), ({3: 63}, IA), ({4: None}, IA), ({5: 63}, IA), ({6: None}, IA),
        ({7: 63}, IA), ({7: 72}, IA), ({5: 72}, IA), ({10: 2}, IA), ({11: -1.0}, IA), ({11: float("nan")}, IA), ({12: 2}, IA),
        ({13: 4}, IA), ({14: 33}, IA), ({15: None, 17: None, 18: None}, IA), ({17: None}, IA), ({15: None}, IA), ({16: 63}, IA),
        ({19: 63}, IA), ({22: None}, IA), ({25: None}, IA), ({23: 2}, IA), ({26: 3}, IA), ({2: 48, 24: 48}, IA),
        ({0: off(1)}, AL), ({4: off(1)}, AL), ({6: off(1)}, AL), ({4: off(8)}, AL), ({6: off(8)}, AL),
        ({0: off(2048), 4: off(4096), 7: 66}, AL), ({17: off(2)}, AL), ({18: off(1)}, AL), ({25: off(2)}, AL), ({8: off(2)}, AL),
        ({1: 1 << 30, 26: 1 << 30}, UN), ({2: 16416, 3: 16416, 5: 16416, 7: 16416, 16: 16416, 19: 16416, 24: 16416}, UN)])


def test_add_norm_backward(fp8):
    #       ds ld  dy r  c   ld  s  ld  g  w  m  rs k  dx ld  dg db ws bytes    st
    #       0  1   2  3  4   5   6  7   8  9  10 11 12 13 14  15 16 17 18       19
    good = [A, 64, A, 4, 64, 64, A, 64, A, 0, A, A, 0, A, 64, A, A, A, 4 * 512, None]
    refuse(fp8, "fp8_add_norm_backward", good, [
        ({0: None}, IA), ({1: 63}, IA), ({2: None}, IA), ({6: None}, IA), ({13: None}, IA), ({11: None}, IA), ({10: None}, IA),
        ({4: 0}, IA), ({5: 60}, IA), ({7: 60}, IA), ({14: 60}, IA), ({14: 72}, IA), ({9: 3}, IA), ({12: -1}, IA), ({17: None}, IA),
        ({18: 2047}, IA), ({0: off(1)}, AL), ({2: off(1)}, AL), ({6: off(1)}, AL), ({13: off(1)}, AL), ({11: off(1)}, AL),
        ({17: off(4)}, AL), ({3: 1 << 30}, UN), ({4: 1 << 27, 1: 1 << 27, 5: 1 << 27, 7: 1 << 27, 14: 1 << 27}, UN)])


def test_mx_add_norm_backward(fp8):
    #       ds ld  dy r  c   ld  xq f  ld  xs ls g  b  w  rs k  dx ld  dg db y  ld  ws bytes    st
    #       0  1   2  3  4   5   6  7  8   9  10 11 12 13 14 15 16 17  18 19 20 21  22 23       24
    good = [A, 64, A, 4, 64, 64, A, 0, 64, A, 4, A, A, 0, A, 0, A, 64, A, A, A, 64, A, 4 * 512, None]
    refuse(fp8, "fp8_mx_add_norm_backward", good, [
        ({0: None}, IA), ({1: 63}, IA), ({6: None}, IA), ({7: 2}, IA), ({9: None}, IA), ({10: 3}, IA), ({14: None}, IA),
        ({17: 72}, IA), ({21: 60}, IA), ({23: 2047}, IA), ({4: 48}, IA), ({0: off(8)}, AL), ({0: off(4096), 1: 66}, AL),
        ({6: off(4)}, AL), ({9: off(2)}, AL), ({20: off(2)}, AL), ({3: 1 << 30, 10: 1 << 30}, UN)])


def test_gemm_swiglu(fp8):
    #       a  fa lda b  fb ldb m  I   k   sa am sb bm act ld  h  ldh  st
    #       0  1  2   3  4  5   6  7   8   9  10 11 12 13 14   15 16   17
    good = [A, 0, 64, A, 0, 64, 4, 32, 64, A, 1, A, 1, A, 32, A, 64, None]
    refuse(fp8, "fp8_gemm_swiglu", good, [
        ({0: None}, IA), ({3: None}, IA), ({1: 4}, IA), ({4: -1}, IA), ({2: 48}, IA), ({5: 48}, IA), ({6: -1}, IA), ({7: -1}, IA),
        ({8: 72, 2: 96, 5: 96}, IA), ({8: -16}, IA), ({9: None}, IA), ({11: None}, IA), ({10: 2}, IA), ({12: -1}, IA),
        ({13: None}, IA), ({14: 31}, IA), ({16: 63}, IA), ({0: off(8)}, AL), ({3: off(8)}, AL), ({2: 72}, AL), ({5: 72}, AL),
        ({9: off(2)}, AL), ({11: off(1)}, AL), ({13: off(1)}, AL), ({15: off(1)}, AL), ({1: 2}, UN), ({4: 3}, UN),
        ({6: 1 << 30}, UN), ({7: 1 << 24, 14: 1 << 24, 16: 1 << 25}, UN), ({6: 1 << 24, 7: 1 << 20, 14: 1 << 20, 16: 1 << 21}, UN),
        ({2: 1 << 24}, UN), ({5: 1 << 24}, UN), ({14: 1 << 25}, UN), ({16: 1 << 25}, UN)])


def test_gemm_swiglu_backward(fp8):
    #       a  fa lda b  fb ldb m  I   k   sa am sb bm h  ldh dh ld  act ld  st
    #       0  1  2   3  4  5   6  7   8   9  10 11 12 13 14  15 16  17 18   19
    good = [A, 0, 64, A, 0, 64, 4, 32, 64, A, 1, A, 1, A, 64, A, 64, A, 32, None]
    refuse(fp8, "fp8_gemm_swiglu_backward", good, [
        ({0: None}, IA), ({3: None}, IA), ({1: 4}, IA), ({2: 48}, IA), ({6: -1}, IA), ({8: 8}, IA), ({9: None}, IA), ({12: 2}, IA),
        ({13: None}, IA), ({15: None}, IA), ({14: 63}, IA), ({16: 63}, IA), ({18: 31}, IA), ({0: off(8)}, AL), ({5: 72}, AL),
        ({13: off(1)}, AL), ({15: off(1)}, AL), ({17: off(1)}, AL), ({4: 2}, UN), ({6: 1 << 30}, UN), ({2: 1 << 24}, UN),
        ({5: 1 << 24}, UN), ({14: 1 << 25}, UN), ({16: 1 << 25}, UN), ({18: 1 << 25}, UN)])


def test_lora_add(fp8):
    ws = fp8.lib.fp8_lora_workspace(4, 16)
    assert ws == 4 * 16 * 16 * 4 and fp8.lib.fp8_lora_workspace(10000, 8) == 10000 * 8 * 4
    assert fp8.lib.fp8_lora_workspace(600, 8) == 8192 * 8 * 4
    assert all(fp8.lib.fp8_lora_workspace(t, r) == 0 for t, r in ((0, 16), (-1, 16), (4, 0), (4, 12), (4, 136)))
    #       x  T  k   ldx idx a  ld  str   b  ld  str  sc E  r   n   base ld out ld  ws bytes st
    #       0  1  2   3   4  5  6   7     8  9   10   11 12 13  14  15 16  17 18  19 20  21
    good = [A, 4, 64, 64, A, A, 64, 1024, A, 16, 512, A, 3, 16, 32, A, 32, A, 32, A, ws, None]
    refuse(fp8, "fp8_lora_add", good, [
        ({0: None}, IA), ({1: -1}, IA), ({2: 0}, IA), ({2: 60, 3: 64}, IA), ({3: 56}, IA), ({4: None}, IA), ({5: None}, IA),
        ({6: 56}, IA), ({7: -8}, IA), ({8: None}, IA), ({9: 8}, IA), ({10: -8}, IA), ({11: None}, IA), ({12: 0}, IA), ({13: 0}, IA),
        ({13: 12}, IA), ({13: 136}, IA), ({14: -1}, IA), ({16: 31}, IA), ({16: 40}, IA), ({17: None}, IA), ({18: 31}, IA),
        ({19: None}, IA), ({20: ws - 1}, IA), ({0: off(8)}, AL), ({3: 68}, AL), ({5: off(2)}, AL), ({6: 68}, AL), ({7: 1028}, AL),
        ({8: off(8)}, AL), ({9: 20}, AL), ({10: 516}, AL), ({15: off(1)}, AL), ({17: off(1)}, AL), ({4: off(2)}, AL),
        ({11: off(1)}, AL), ({19: off(8)}, AL), ({1: 1 << 25}, UN), ({14: 1 << 24, 16: 1 << 24, 18: 1 << 24}, UN),
        ({3: 1 << 24}, UN), ({6: 1 << 24}, UN), ({9: 1 << 24}, UN), ({16: 1 << 24, 18: 1 << 24}, UN),
        ({15: off(1 << 16), 16: 1 << 24}, UN), ({15: None, 18: 1 << 24}, UN)])


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def f32(*shape):
    return torch.zeros(shape)


def bad(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_python_add_norm(fp8):
    n = fp8.fp8_add_norm_quantize_row
    args = lambda **k: dict(dict(x=bf(4, 64), res=bf(4, 64), sum_out=bf(4, 64), gamma=bf(64), beta=None, eps=1e-5,  # noqa: E731
                                 kind=1, fmt=0, margin=0, q=u8(4, 64), scale_inv_out=f32(4)), **k)
    bad("on a GPU", n, **args())
    bad("res must be", n, **args(res=bf(4, 32)))
    bad("res must be torch.bfloat16", n, **args(res=f32(4, 64)))
    bad("sum_out must be", n, **args(sum_out=bf(3, 64)))
    bad("rows overlap", n, **args(res=bf(64).expand(4, 64)))
    bad("gamma", n, **args(gamma=bf(32)))
    bad("scale_inv_out", n, **args(scale_inv_out=f32(3)))
    b = fp8.fp8_add_norm_backward
    back = lambda **k: dict(dict(dsum=bf(4, 64), dy=bf(4, 64), sum=bf(4, 64), gamma=None, mean=f32(4), rstd=f32(4),  # noqa: E731
                                 kind=0, dx=bf(4, 64)), **k)
    bad("on a GPU", b, **back())
    bad("dsum must be", b, **back(dsum=bf(4, 32)))
    bad("sum must be", b, **back(sum=bf(5, 64)))
    bad("dx must be", b, **back(dx=bf(4, 32)))
    m = fp8.fp8_mx_add_norm_backward
    bad("on a GPU", m, bf(4, 64), bf(4, 64), u8(4, 64), 0, u8(1, 4, 4), None, None, f32(4), 0, bf(4, 64))
    bad("dsum must be", m, bf(4, 32), bf(4, 64), u8(4, 64), 0, u8(1, 4, 4), None, None, f32(4), 0, bf(4, 64))


def test_python_glu(fp8):
    g = fp8.fp8_gemm_swiglu
    args = lambda **k: dict(dict(a=u8(4, 64), fa=0, b=u8(32, 64), fb=0, a_scale_inv=f32(4), a_mode=1,  # noqa: E731
                                 b_scale_inv=f32(32), b_mode=1, act=bf(4, 16)), **k)
    bad("on a GPU", g, **args())
    bad("b must be", g, **args(b=u8(32, 48)))
    bad("b must be", g, **args(b=u8(31, 64)))
    bad("act must be", g, **args(act=bf(4, 32)))
    bad("h must be", g, **args(h=bf(4, 16)))
    bad("a_scale_inv", g, **args(a_scale_inv=f32(1)))
    bad("a_scale_inv", g, **args(a_mode=0))
    bad("b_scale_inv", g, **args(b_scale_inv=f32(16)))
    bad("rows overlap", g, **args(a=u8(64).expand(4, 64)))
    b = fp8.fp8_gemm_swiglu_backward
    back = lambda **k: dict(dict(a=u8(4, 64), fa=0, b=u8(16, 64), fb=0, a_scale_inv=f32(4), a_mode=1,  # noqa: E731
                                 b_scale_inv=f32(16), b_mode=1, h=bf(4, 32), dh=bf(4, 32)), **k)
    bad("on a GPU", b, **back())
    bad("h must be", b, **back(h=bf(4, 16)))
    bad("dh must be", b, **back(dh=bf(4, 16)))
    bad("act must be", b, **back(act=bf(4, 32)))
    bad("k = 64", b, **back(b=u8(16, 48)))


def test_python_lora(fp8):
    lo = fp8.fp8_lora_add
    args = lambda **k: dict(dict(x=bf(4, 64), lora_a=bf(3, 16, 64), lora_b=bf(3, 32, 16), scaling=f32(3),  # noqa: E731
                                 adapter_idx=torch.zeros(4, dtype=torch.int32), base=bf(4, 32), out=bf(4, 32),
                                 workspace=f32(4096)), **k)
    bad("on a GPU", lo, **args())
    bad("do not match", lo, **args(lora_a=bf(3, 16, 32)))
    bad("do not match", lo, **args(lora_b=bf(2, 32, 16)))
    bad("do not match", lo, **args(lora_b=bf(3, 32, 8)))
    bad("lora_a must be", lo, **args(lora_a=bf(16, 64)))
    bad("rows overlap", lo, **args(lora_b=bf(3, 1, 16).expand(3, 32, 16)))
    bad("scaling", lo, **args(scaling=f32(4)))
    bad("adapter_idx", lo, **args(adapter_idx=torch.zeros(4, dtype=torch.int64)))
    bad("adapter_idx", lo, **args(adapter_idx=torch.zeros(5, dtype=torch.int32)))
    bad("base must be", lo, **args(base=bf(4, 16)))
    bad("out must be", lo, **args(out=bf(3, 32)))


@pytest.mark.parametrize("source", ["gemm_swiglu.hip", "lora.hip"])
def test_no_scratch(source):
    out = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-ffp-contract=off", "-Xclang",
                          "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S", "-o", "-",
                          os.path.join(CSRC, source)], capture_output=True, text=True)
    assert out.returncode == 0, out.stderr[-2000:]
    sizes = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", out.stdout)
    assert sizes and all(int(s) == 0 for s in sizes), "a kernel uses scratch memory"
    assert "scratch_" not in out.stdout


@pytest.mark.parametrize("source", ["gemm_swiglu.hip", "lora.hip"])
def test_no_warnings(source):
    out = subprocess.run([HIPCC, "--offload-arch=gfx950", "-std=c++17", "-ffp-contract=off", "-Wall", "-Werror",
                          "-Wno-unused-command-line-argument", "-Xclang", "-target-feature", "-Xclang",
                          "-packed-fp32-ops", "--cuda-device-only", "-O1", "-c", "-o", os.devnull,
                          os.path.join(CSRC, source)], capture_output=True, text=True)
    assert out.returncode == 0 and "warning" not in out.stderr, out.stderr[-3000:]


def test_m0_only_feeds_direct_loads():
    """In the gated products' kernels M0 is only the LDS base of direct loads, with the
    wait states that an assembly statement has to bring along."""
    from test_isa_guards import kernels
    out = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-ffp-contract=off", "-Xclang",
                          "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S", "-o", "-",
                          os.path.join(CSRC, "gemm_swiglu.hip")], capture_output=True, text=True)
    assert out.returncode == 0, out.stderr[-2000:]
    found, loads = kernels(out.stdout), 0
    for name, body in found.items():
        lines = [l.strip() for l in body.splitlines() if l.strip() and not l.strip().startswith(";")]
        for i, l in enumerate(lines):
            if re.search(r"\bm0\b", l):
                assert re.match(r"s_mov_b32 m0, (s\d+|vcc_lo|vcc_hi)$", l), (name, l)
                assert lines[i + 1] in ("s_nop 0", "s_nop 4"), (name, l)
                m = re.match(r"global_load_lds_dword(x4)? v\S+, (off|s\[\d+:\d+\]|vcc)$", lines[i + 2])
                assert m and (m.group(2) == "off" or lines[i + 1] == "s_nop 4"), (name, lines[i + 2])
                loads += 1
    assert loads > 0

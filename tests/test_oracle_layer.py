"""Pins of oracle/layer.py, the fp64 definitions of the layer around the FP8
products: rows worked by hand, gradients against differences of the forward
pass, invariants."""
import numpy as np
import pytest

import workloads
from oracle import layer


def test_norm_row_by_hand():
    # 1, 2, 3, 4: mean 2.5, variance 1.25; RMS: mean square 7.5
    x = np.array([[1.0, 2.0, 3.0, 4.0]])
    f = layer.norm_forward(x, np.array([2.0, 1, 1, 1]), np.array([0.0, 0, 0, 1]), 0.0, False)
    assert f["mean"][0] == 2.5
    assert np.isclose(f["rstd"][0], 1 / np.sqrt(1.25), rtol=1e-15)
    assert np.allclose(f["y"][0], np.array([-3.0, -0.5, 0.5, 1.5]) / np.sqrt(1.25) + [0, 0, 0, 1], rtol=1e-15)
    f = layer.norm_forward(x, None, None, 0.25, True)
    assert f["mean"][0] == 0 and np.isclose(f["rstd"][0], 1 / np.sqrt(7.75), rtol=1e-15)
    assert np.allclose(f["y"], x / np.sqrt(7.75), rtol=1e-15)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradient_against_differences(rms):
    rng = np.random.default_rng(1 + rms)
    x, dy = rng.standard_normal((3, 12)), rng.standard_normal((3, 12))
    gamma, beta, eps, h = rng.standard_normal(12), rng.standard_normal(12), 0.1, 1e-5

    def loss(x, gamma, beta):
        return (layer.norm_forward(x, gamma, beta, eps, rms)["y"] * dy).sum()

    f = layer.norm_forward(x, gamma, beta, eps, rms)
    b = layer.norm_backward(dy, f["xhat"], gamma, f["rstd"], rms)
    for r in range(3):
        for c in range(12):
            e = np.zeros_like(x)
            e[r, c] = h
            d = (loss(x + e, gamma, beta) - loss(x - e, gamma, beta)) / (2 * h)
            assert abs(d - b["dx"][r, c]) < 1e-8        # (third derivative h^2 / 6, differences' rounding 1e-11)
    for c in range(12):
        e = np.zeros(12)
        e[c] = h
        assert abs((loss(x, gamma + e, beta) - loss(x, gamma - e, beta)) / (2 * h) - b["dgamma"][c]) < 1e-8
        assert abs((loss(x, gamma, beta + e) - loss(x, gamma, beta - e)) / (2 * h) - b["dbeta"][c]) < 1e-8


def test_norm_gradient_invariants():
    """The layer norm's output does not see a constant added to the row nor (eps = 0)
    its scale: dx sums to 0 and is orthogonal to x."""
    rng = np.random.default_rng(3)
    x, dy = rng.standard_normal((5, 40)), rng.standard_normal((5, 40))
    f = layer.norm_forward(x, None, None, 0.0, False)
    dx = layer.norm_backward(dy, f["xhat"], None, f["rstd"], False)["dx"]
    assert np.abs(dx.sum(1)).max() < 1e-13 and np.abs((dx * x).sum(1)).max() < 1e-12


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(4)
    g, u, da, h = rng.standard_normal(50) * 4, rng.standard_normal(50), rng.standard_normal(50), 1e-5
    b = layer.swiglu_backward(da, g, u)
    fwd = lambda g, u: layer.swiglu(g, u)[0] * da  # noqa: E731
    assert np.allclose((fwd(g + h, u) - fwd(g - h, u)) / (2 * h), b["dg"], atol=1e-8)
    assert np.allclose((fwd(g, u + h) - fwd(g, u - h)) / (2 * h), b["du"], atol=1e-8)
    z = layer.swiglu_backward(np.ones(1), np.zeros(1), np.full(1, 3.0))
    assert z["dg"][0] == 1.5 and z["du"][0] == 0 and z["a"][0] == 0


def test_checkpoint_values_undo_the_cast(orc):
    """mx_values of mx_quantize_row is within half a step of the input (the largest
    codes saturate: at most 1/8 below)."""
    rng = np.random.default_rng(5)
    x = workloads.bf16_bits((rng.standard_normal((9, 96)) * np.exp2(rng.integers(-9, 9, (9, 1)))).astype(np.float32))
    for fmt in (orc.E4M3, orc.E5M2):
        q, s = orc.mx_quantize_row(x, fmt)
        v = layer.values(x)
        got = layer.mx_values(q, fmt, s)
        scale = np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=1)
        sat = np.abs(v) / scale > orc.fmt_info(fmt)[0]
        assert np.all(np.abs(got - v)[~sat] <= (layer.half_step(fmt, v / scale) * scale)[~sat])
        assert np.all(np.abs(got - v)[sat] <= np.abs(v)[sat] / 8)
        layer.checkpoint_ok(fmt, q, s, v, np.zeros_like(v))


def test_records_round_trip():
    s = np.arange(2 * 5, dtype=np.uint8).reshape(2, 5) + 100          # 160 columns: two records, three spare bytes
    rec = np.zeros((2, 2, 4), np.uint8)
    for r in range(2):
        for b in range(5):
            rec[b // 4, r, b % 4] = s[r, b]
    assert np.array_equal(layer.from_records(rec, 160), s)


def test_cast_check_sees_a_wrong_code(orc):
    rng = np.random.default_rng(6)
    x = workloads.bf16_bits(rng.standard_normal((4, 64)).astype(np.float32))
    q, si, _ = orc.quantize_row(x, orc.E4M3)
    v = layer.values(x)
    layer.cast_ok(orc.E4M3, q, si, v, np.zeros_like(v))
    q[2, 3] += 1
    with pytest.raises(AssertionError):
        layer.cast_ok(orc.E4M3, q, si, v, np.zeros_like(v))


def test_moe_few_by_hand():
    """One token, two slots: expert 1 twice and an index out of range."""
    x = np.array([[1.0, 2.0]])
    w1 = np.zeros((2, 2, 2))
    w1[1] = [[3.0, 0.0], [0.0, 1.0]]                    # gate 3, up 2
    w2 = np.zeros((2, 2, 1))
    w2[1] = [[1.0], [-1.0]]
    out, _ = layer.moe_few(x, np.array([[1, 1, 5]]), np.array([[0.25, 0.5, 9.0]]), w1, w2)
    a = 3.0 / (1 + np.exp(-3.0)) * 2.0 * 0.75
    assert np.allclose(out, [[a, -a]], rtol=1e-14)

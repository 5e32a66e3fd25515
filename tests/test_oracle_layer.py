"""Pins of the oracle of the operators around a quantized layer."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import layer


def test_codes_reconstruct_within_half_a_step():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 77)) * np.exp(rng.uniform(-20, 20, (40, 1)))).astype(np.float32)
    q, s = layer.quantize_rows(x)
    amax = np.abs(x).max(1).astype(np.float64)
    assert (np.abs(q.astype(int)).max(1) == 127).all()
    # scale and 127/amax each carry one rounding: 127 codes of relative error 2^-23 on top of half a step
    err = np.abs(q * s[:, None].astype(np.float64) - x)
    assert (err <= amax[:, None] / 127 * (0.5 + 127 * 2.0 ** -22)).all()


def test_codes_of_special_rows():
    x = np.zeros((6, 5), np.float32)
    x[1, 2] = np.inf
    x[2, 3] = np.nan
    x[3, 0] = 1e-35
    x[4] = [1, -1, 0.5, 0, -0.5]
    x[5, 1] = 3.4028235e38
    q, s = layer.quantize_rows(x)
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] == 0 and np.isfinite(s[5])
    assert not q[:4].any()
    assert q[4].tolist() == [127, -127, 64, 0, -64] and q[5].tolist() == [0, 127, 0, 0, 0]


def test_product_is_the_exact_sum_scaled_in_three_roundings():
    rng = np.random.default_rng(2)
    a = rng.integers(-128, 128, (3, 91)).astype(np.int8)
    b = rng.integers(-128, 128, (4, 91)).astype(np.int8)
    sa = rng.uniform(0.01, 1, 3).astype(np.float32)
    sb = rng.uniform(0.01, 1, 4).astype(np.float32)
    bias = rng.standard_normal(4).astype(np.float32)
    got = layer.product(a, sa, b, sb, bias)
    for m in range(3):
        for n in range(4):
            exact = sum(int(x) * int(y) for x, y in zip(a[m], b[n]))
            v = Fraction(exact) * Fraction(float(sa[m])) * Fraction(float(sb[n]))
            want = float(v + Fraction(float(bias[n])))
            assert abs(got[m, n] - want) <= 2.0 ** -24 * (2.1 * abs(float(v)) + abs(want)) * 1.01


@pytest.mark.parametrize("rot", [2, 4, 64, 128])
def test_frequencies(rot):
    f, amp = layer.frequencies(rot)
    assert amp == 1.0 and f[0] == 1.0
    assert np.allclose(f, [10000.0 ** (-2 * i / rot) for i in range(rot // 2)], rtol=1e-14)
    lin, _ = layer.frequencies(rot, scaling="linear", factor=4.0)
    assert np.allclose(lin * 4, f, rtol=1e-15)
    ntk, _ = layer.frequencies(rot, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0
    if rot > 2:
        assert np.isclose(ntk[-1], f[-1] / 4.0, rtol=1e-12)  # the lowest frequency is divided by the factor
    yarn, amp = layer.frequencies(rot, scaling="yarn", factor=4.0, original_length=8192)
    turns = 8192 * f / (2 * np.pi)
    assert np.allclose(yarn[turns >= 32], f[turns >= 32], rtol=1e-14)
    assert np.allclose(yarn[turns <= 1], f[turns <= 1] / 4, rtol=1e-14)
    assert (yarn <= f * (1 + 1e-14)).all() and (yarn >= f / 4 * (1 - 1e-14)).all()
    assert np.isclose(amp, 1 + 0.1 * np.log(4.0))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_is_a_complex_product(layout):
    rng = np.random.default_rng(3)
    T, H, D, rot = 5, 3, 20, 12
    x = rng.standard_normal((T, H, D))
    f, _ = layer.frequencies(rot)
    ang = np.arange(50)[:, None] * f
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    pos = rng.integers(0, 50, T)
    y = layer.rotate(x, pos, table, layout, dtype=np.float64)
    ia, ib = layer.pairs(rot, layout)
    z = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * ang[pos])[:, None, :]
    assert np.allclose(y[..., ia], z.real, atol=1e-13) and np.allclose(y[..., ib], z.imag, atol=1e-13)
    assert np.array_equal(y[..., rot:], x[..., rot:])
    back = layer.rotate(y, pos, table, layout, inverse=True, dtype=np.float64)
    assert np.allclose(back, x, atol=1e-13)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradients_against_central_differences(layout):
    rng = np.random.default_rng(4)
    T, H, D, rot, eps = 3, 2, 10, 6, 1e-3
    x, g = rng.standard_normal((2, T, H, D))
    w = rng.standard_normal(D)
    f, _ = layer.frequencies(rot)
    ang = np.arange(9)[:, None] * f
    table = 1.2 * np.concatenate([np.cos(ang), np.sin(ang)], 1)
    pos = np.array([0, 8, 3])

    def loss(x, w):
        return (layer.norm_rope(x, w, pos, table, eps, layout)[0] * g).sum()

    dx, _, dw, _ = layer.norm_rope_back(g, x, w, pos, table, eps, layout)
    h = 1e-6
    for idx in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[idx] = h
        # central difference: truncation h^2 / 6 times the third derivative, rounding 2^-52 |loss| / h
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - dx[idx]) < 1e-8
    for i in range(D):
        d = np.zeros(D)
        d[i] = h
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - dw[i]) < 1e-8


def test_append_skips_padding_and_slots_outside():
    cache = np.arange(2 * 3 * 1 * 2, dtype=np.float32).reshape(2, 3, 1, 2)
    rows = -np.ones((4, 1, 2), np.float32)
    out = layer.append(cache, rows, [4, -1, 6, 0])
    assert (out[1, 1] == -1).all() and (out[0, 0] == -1).all()
    keep = np.ones((2, 3), bool)
    keep[1, 1] = keep[0, 0] = False
    assert np.array_equal(out[keep], cache[keep])

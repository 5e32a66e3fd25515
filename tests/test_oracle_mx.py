"""Pins of the MXFP4 and layer norm oracle: codes against exact rationals,
gradients against central differences."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import mx

MAGNITUDES = [Fraction(n, 2) for n in (0, 1, 2, 3, 4, 6, 8, 12)]


def nearest(v, scale):
    """Code of the nearest level, ties to the even code, by search."""
    y = abs(Fraction(float(v))) / scale
    return min(range(8), key=lambda i: (abs(MAGNITUDES[i] - y), i % 2)) + (8 if np.signbit(v) else 0)


@pytest.mark.parametrize("kind", ["normal", "ties", "tiny", "huge", "spread"])
def test_codes_are_nearest(kind):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((3, 70)).astype(np.float32)
    if kind == "ties":
        x = (rng.integers(-32, 33, x.shape) * 0.25).astype(np.float32)
    elif kind == "tiny":
        x = (rng.integers(-9, 10, x.shape) * 2.0 ** -149).astype(np.float32)
    elif kind == "huge":
        x = (x * 2.0 ** 124).clip(-3.4e38, 3.4e38).astype(np.float32)
    elif kind == "spread":
        x = (x * np.exp2(rng.integers(-40, 40, x.shape))).astype(np.float32)
    codes, scales = mx.quantize(x)
    assert codes.shape == (3, 48) and scales.shape == (3, 3)
    for r in range(3):
        for b in range(3):
            block = x[r, 32 * b:32 * b + 32]
            top = Fraction(float(np.abs(block).max()))
            e = -127
            if top:
                while Fraction(2) ** (e + 3) <= top:
                    e += 1
            assert int(scales[r, b]) == e + 127
            for i, v in enumerate(block):
                at = 32 * b + i
                code = codes[r, at // 2] >> (4 * (at % 2)) & 15
                assert code == nearest(v, Fraction(2) ** e), (v, e)
    assert (codes[:, 35:] == 0).all()  # values past the row


def test_blocks_that_are_not_finite():
    x = np.ones((2, 96), np.float32)
    x[0, 5], x[1, 95] = np.nan, -np.inf
    codes, scales = mx.quantize(x)
    assert scales.tolist() == [[255, 125, 125], [125, 125, 255]]
    assert not codes[0, :16].any() and not codes[1, 32:].any() and (codes[0, 16:] == 0x66).all()
    v = mx.values(codes, scales)
    assert np.isnan(v[0, :32]).all() and (v[0, 32:] == 1).all()


def test_values_of_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 16))
    for s in (0, 1, 127, 254):
        v = mx.values(codes, np.full((256, 1), s, np.uint8))
        for c in (0, 0x17, 0xF8, 255):
            lo, hi = c & 15, c >> 4
            assert Fraction(float(v[c, 0])) == MAGNITUDES[lo & 7] * (-1 if lo & 8 else 1) * Fraction(2) ** (s - 127)
            assert Fraction(float(v[c, 1])) == MAGNITUDES[hi & 7] * (-1 if hi & 8 else 1) * Fraction(2) ** (s - 127)


def test_linear_backward_is_the_gradient_of_the_rounded_operands():
    # with operands that MXFP4 holds exactly, the gradients of sum(dout * (X W^T + b))
    rng = np.random.default_rng(4)
    M, N, K = 6, 5, 7
    dout, x, w = (rng.choice([-3.0, -1.0, -0.5, 0.5, 1.0, 2.0, 6.0], s).astype(np.float32) for s in ((M, N), (M, K), (N, K)))
    (dx, _), (dw, _), (db, _) = mx.linear_backward(dout, x, w)
    for got, v in ((dx, x), (dw, w)):
        for i in np.ndindex(v.shape):
            up, down = v.astype(np.float64), v.astype(np.float64)
            up[i] += 0.5
            down[i] -= 0.5
            f = [float((dout * (a @ w.T if v is x else x @ a.T)).sum()) for a in (up, down)]
            assert got[i] == f[0] - f[1]
    assert np.array_equal(db, dout.sum(0))


@pytest.mark.parametrize("d,eps", [(1, 1e-5), (2, 1e-5), (7, 0.1), (40, 1e-5)])
def test_layer_norm_gradient_against_differences(d, eps):
    rng = np.random.default_rng(d)
    x, g = rng.standard_normal((3, d)) + 2, rng.standard_normal((3, d))
    w, b = rng.standard_normal(d), rng.standard_normal(d)

    def f(x, w, b):
        return float((g * mx.layer_norm(x, w, b, eps)[0]).sum())
    grads = [v for v, _ in mx.layer_norm_back(g, x, w, eps)]
    at = [x, w, b]
    for k in range(3):
        for i in np.ndindex(at[k].shape):
            step = 1e-5
            hi, lo = [v.copy() for v in at], [v.copy() for v in at]
            hi[k][i] += step
            lo[k][i] -= step
            # central differences: h^2 f''' / 6 of the third derivative (at most r^3 ~ 1e4 here for d = 2), and rounding
            want = (f(*hi) - f(*lo)) / (2 * step)
            assert abs(grads[k][i] - want) <= 1e-5 * (1 + abs(want)), (k, i)


def test_layer_norm_values():
    y, _ = mx.layer_norm([[1.0, 2.0, 3.0]], [1.0, 1.0, 2.0], [0.0, 0.0, 5.0], 0.0)
    s = np.sqrt(1.5)
    assert np.allclose(y, [[-s, 0.0, 5.0 + 2 * s]], rtol=0, atol=1e-15)

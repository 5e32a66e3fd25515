"""Microscaled 4-bit (MXFP4) codes, their product and its gradients, and the
layer norm with its gradients.

Test infrastructure only.  Codes and scales are defined bit for bit and are
restated in exact arithmetic (every step below is exact in float64, or on
integers).  Products and norms leave the order of their sums open: they are
computed in float64, next to the bound that an fp32 evaluation has to keep.

The bounds, with u = 2^-24 the error of one rounded fp32 operation and g(n) =
n u / (1 - n u):

* product: each product of two codes with its scales is exact (4 significant
  bits), a sum of n of them in any order is within g(n) of the sum of their
  magnitudes where every addition rounds to nearest; a matrix core that truncates
  is within twice that.  The bias is one addition more.
* norm: a sum that is taken in a tree of depth D is within g(D) of the sum of
  magnitudes.  With c = x - mean, m1 the distance of the rounded mean from it
  and A = mean|c| + |m1|, the centred value x - m0 - m1 has two roundings and
  the error of m1: at most g(D + 6) (|c| + A).  mean((x - m0)^2) - m1^2 is within
  g(D + 6) (var + 3 m1^2) of var, so r = 1 / sqrt(var + eps) within half of that
  over (var + eps), plus 3 u, relative.  Products with r and w and the sum with b are
  4 roundings more.
* its gradient: the same for xh = c r, with e its bound.  mean(h) is within g(D + 3)
  of mean|h|, mean(h xh) within g(D + 4) of mean|h xh| plus mean(|h| e).  dw and db
  are sums over rows in any order: g(rows + 4) of the sum of magnitudes, plus
  the sum of |dy| e for dw.

Parity: pinned in ``tests/test_oracle_mx.py`` (codes against exact rationals,
gradients against central differences).
"""

import numpy as np

from .layer import U, gamma

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# --------------------------------------------------------------------------
# codes
# --------------------------------------------------------------------------
def blocks(d):
    return -(-d // 32)


def quantize(x32):
    """(codes uint8 [rows, 16 blocks], scale bytes [rows, blocks]) of fp32 rows."""
    x = np.asarray(x32, np.float32)
    rows, d = x.shape
    b = np.zeros((rows, blocks(d) * 32), np.float32)
    b[:, :d] = x
    b = b.reshape(rows, -1, 32)
    exponent = ((b.view(np.uint32) >> 23) & 255).astype(np.int64).max(-1)  # of the largest magnitude
    byte = np.where(exponent == 255, 255, np.maximum(exponent - 2, 0)).astype(np.uint8)
    with np.errstate(invalid="ignore"):
        y = np.abs(b).astype(np.float64) / np.exp2(byte.astype(np.float64) - 127.0)[..., None]
    code = np.zeros(y.shape, np.uint8)
    for i in range(7):  # past the middle between two levels, or on it if the upper code is even
        middle = (LEVELS[i] + LEVELS[i + 1]) / 2
        code += (y >= middle) if i % 2 else (y > middle)
    code += 8 * np.signbit(b).astype(np.uint8)
    code[byte == 255] = 0
    code = code.reshape(rows, -1, 2)
    return (code[..., 0] | code[..., 1] << 4).astype(np.uint8), byte


def values(codes, scales, d=None):
    """float64 values of codes and scales."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1, 32)
    v = LEVELS[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.exp2(scales.astype(np.float64) - 127.0)
    s[scales == 255] = np.nan
    v = (v * s[..., None]).reshape(codes.shape[0], -1)
    return v if d is None else v[:, :d]


def rounded(x32):
    """float64 values that the rows' codes stand for."""
    x = np.asarray(x32, np.float32)
    return values(*quantize(x), x.shape[1])


# --------------------------------------------------------------------------
# product
# --------------------------------------------------------------------------
def product(x, w, bias=None):
    """(float64 x w^T + bias, its bound) of values."""
    n = x.shape[1] + (bias is not None)
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    return y, 2 * gamma(n) * mag


def linear_backward(dout, x, w):
    """((dX, bound), (dW, bound), (db, bound)) of fp32 values."""
    dout, x, w = (np.asarray(v, np.float32) for v in (dout, x, w))
    t = np.ascontiguousarray
    dx = product(rounded(dout), rounded(t(w.T)))
    dw = product(rounded(t(dout.T)), rounded(t(x.T)))
    g = dout.astype(np.float64)
    return dx, dw, (g.sum(0), gamma(g.shape[0]) * np.abs(g).sum(0))


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------
def _depth(d):
    """Of the sums over a row: a thread's own elements, 6 steps in a wave, 16
    waves; rows that stay in registers have at most 64 elements a thread."""
    return 96 + d // 1024


def _center(x, eps):
    """c, r, bound of the centred value, relative bound of r."""
    d = x.shape[1]
    D = _depth(d)
    mean = x.mean(1, keepdims=True)
    c = x - mean
    m1 = gamma(D + 1) * np.abs(x).mean(1, keepdims=True)
    var = (c * c).mean(1, keepdims=True)
    r = 1.0 / np.sqrt(var + eps)
    e = gamma(D + 6) * (np.abs(c) + np.abs(c).mean(1, keepdims=True) + m1)
    er = 0.5 * gamma(D + 6) * (var + 3 * m1 * m1) / (var + eps) + 3 * U
    return c, r, e, er


def layer_norm(x, w, b, eps):
    """(float64 values, bound before the last rounding)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    c, r, e, er = _center(x, eps)
    y = c * r * w
    bound = np.abs(w) * r * (e + np.abs(c) * er)
    mag = np.abs(y)
    if b is not None:
        y, mag = y + np.asarray(b, np.float64), mag + np.abs(np.asarray(b, np.float64))
    return y, 1.01 * bound + gamma(4) * mag


def layer_norm_back(g, x, w, eps):
    """((dx, bound), (dw, bound), (db, bound))."""
    g, x, w = (np.asarray(v, np.float64) for v in (g, x, w))
    rows, d = x.shape
    D = _depth(d)
    c, r, e, er = _center(x, eps)
    xh = c * r
    exh = 1.01 * r * (e + np.abs(c) * er) + 2 * U * np.abs(xh)
    h = g * w

    def mean(v):
        return v.mean(1, keepdims=True)
    mh, mhx = mean(h), mean(h * xh)
    dx = r * (h - mh - xh * mhx)
    emhx = gamma(D + 4) * mean(np.abs(h * xh)) + mean(np.abs(h) * exh)
    bound = r * (gamma(D + 3) * mean(np.abs(h)) + exh * np.abs(mhx) + np.abs(xh) * emhx
                 + 6 * U * (np.abs(h) + np.abs(mh) + np.abs(xh * mhx))) + er * np.abs(dx)
    dw, db = (g * xh).sum(0), g.sum(0)
    edw = gamma(rows + 4) * np.abs(g * xh).sum(0) + (np.abs(g) * exh).sum(0)
    return (dx, 1.01 * bound), (dw, 1.01 * edw), (db, gamma(rows + 4) * np.abs(g).sum(0))

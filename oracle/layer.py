"""The operators around a quantized layer: int8 rows and their product,
rotary positions, head norms with the rotation and their gradient, the paged
append.

Test infrastructure only.  Operators whose every rounding is defined (codes,
integer product with its epilogue, rotation, append) are restated in float32,
one operation at a time, and are compared bit for bit.  The norms leave the
order of their sums open: they are computed in float64, next to the bound an
fp32 evaluation has to keep.

The bounds.  u = 2^-24 is the error of one rounded fp32 operation, g(n) =
n u / (1 - n u).  A sum of n terms in any order is within g(n) of the sum of
their magnitudes.

* forward: mean(x^2) has relative error at most g(D + 2) (squares, sum,
  division), its sqrt half of that plus u, so that the reciprocal root r is
  within g(D/2 + 5); y = x r w adds 2 roundings, the rotation 2 more over
  |a c| + |b s|, c and s are taken as given.  Together g(D/2 + 10) (|a c| +
  |b s|), then one rounding to T.
* backward: u_ = R^T g within g(2) of |g| terms, xhat within g(D/2 + 6);
  the mean of u_ w xhat is within g(D + D/2 + 12) of the mean of magnitudes
  m; dx = r (u_ w - xhat mean) is within g(2 D + 30) r (|u_ w| + |xhat| m).
  dw is a sum of n terms u_ xhat: g(n + D/2 + 12) times the sum of magnitudes.

Parity: pinned in ``tests/test_oracle_layer.py`` (codes and product against
exact integers and rationals, frequencies against their defining properties,
rotation against complex numbers, gradients against central differences).
"""

import numpy as np

from .numerics import to_bf16_bits, widen

U = 2.0 ** -24


def gamma(n):
    return n * U / (1.0 - n * U)


def half_ulp(t):
    """Largest relative error of one rounding to the type, and the largest
    absolute one among its subnormals."""
    return {"fp32": (2.0 ** -24, 2.0 ** -150), "fp16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 2.0 ** -134)}[t]


def round_to(x32, t):
    """fp32 values as the type's raw bits (fp32: the bits themselves)."""
    x32 = np.ascontiguousarray(x32, dtype=np.float32)
    if t == "fp32":
        return x32.view(np.uint32)
    if t == "fp16":
        with np.errstate(over="ignore"):
            return x32.astype(np.float16).view(np.uint16)
    return to_bf16_bits(x32)


def values(bits, t):
    """Raw bits as fp32 values."""
    bits = np.ascontiguousarray(bits)
    if t == "fp32":
        return bits.view(np.float32)
    if t == "fp16":
        return bits.view(np.float16).astype(np.float32)
    return widen(bits, "bf16")


# --------------------------------------------------------------------------
# int8 linear
# --------------------------------------------------------------------------
def quantize_rows(x32):
    """(codes int8, scale fp32) of the rows."""
    x = np.asarray(x32, np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(axis=1)  # NaN if any
        scale = (amax / np.float32(127)).astype(np.float32)
        inv = (np.float32(127) * (np.float32(1) / amax).astype(np.float32)).astype(np.float32)
        tiny = amax < np.float32(2.0 ** -100)
        scale[tiny] = inv[tiny] = 0
        bad = ~np.isfinite(amax)
        scale[bad] = np.nan
        q = np.rint((x * inv[:, None]).astype(np.float32))
        q[bad] = 0
    return q.astype(np.int8), scale


def product(codes, scale, w_codes, w_scale, bias=None):
    """fp32 values before the rounding to T."""
    # integers below 2^31 in every partial sum: exact in fp64, in any order
    acc = codes.astype(np.float64) @ w_codes.astype(np.float64).T
    with np.errstate(all="ignore"):
        v = (acc.astype(np.float32) * scale[:, None]).astype(np.float32)
        v = (v * w_scale[None, :]).astype(np.float32)
        if bias is not None:
            v = (v + bias[None, :]).astype(np.float32)
    return v


# --------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------
def frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_length=0, slow=1.0, fast=32.0):
    i = np.arange(0, rot, 2, dtype=np.float64)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = np.exp(-np.log(base) * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        turns = original_length / (2 * np.pi / f)
        ramp = np.interp(turns, [slow, fast], [0.0, 1.0])
        f = f * ramp + f * (1 - ramp) / factor
    return f, (0.1 * np.log(factor) + 1 if scaling == "yarn" else 1.0)


def pairs(rot, layout):
    """(first, second) element indices of the pairs."""
    i = np.arange(rot // 2)
    return (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)


def rotate(x, positions, table, layout, inverse=False, dtype=np.float32):
    """x [.., tokens, heads, dim]; every operation rounded to dtype."""
    y = np.array(x, dtype=dtype)
    max_pos, rot = table.shape
    pos = np.asarray(positions)
    ok = (pos >= 0) & (pos < max_pos)
    row = table[np.where(ok, pos, 0)].astype(dtype)
    row[~ok] = np.nan
    c, s = row[..., None, :rot // 2], row[..., None, rot // 2:]
    if inverse:
        s = -s
    ia, ib = pairs(rot, layout)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    with np.errstate(all="ignore"):
        y[..., ia] = (a * c).astype(dtype) - (b * s).astype(dtype)
        y[..., ib] = (b * c).astype(dtype) + (a * s).astype(dtype)
    return y


def rotate_magnitude(x, positions, table, layout):
    """|a c| + |b s| of every element (its own magnitude where not rotated)."""
    rot = table.shape[1]
    y = np.abs(np.asarray(x, np.float64))
    row = np.abs(table[np.asarray(positions)].astype(np.float64))
    c, s = row[..., None, :rot // 2], row[..., None, rot // 2:]
    ia, ib = pairs(rot, layout)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c + b * s, b * c + a * s
    return y


# --------------------------------------------------------------------------
# norms with the rotation
# --------------------------------------------------------------------------
def _root(x, eps):
    return 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)


def norm_rope(x, w, positions, table, eps, layout):
    """(float64 values, bound of an fp32 evaluation before its last rounding)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    n = x * _root(x, eps) * w
    y = rotate(n, positions, table, layout, dtype=np.float64)
    return y, gamma(x.shape[-1] / 2 + 10) * rotate_magnitude(n, positions, table, layout)


def norm_rope_back(g, x, w, positions, table, eps, layout):
    """(dx, its bound, dw, its bound) in float64."""
    g, x, w = (np.asarray(v, np.float64) for v in (g, x, w))
    D = x.shape[-1]
    r = _root(x, eps)
    xhat = x * r
    up = rotate(g, positions, table, layout, inverse=True, dtype=np.float64)
    up_mag = rotate_magnitude(g, positions, table, layout)
    inner = np.mean(up * w * xhat, axis=-1, keepdims=True)
    inner_mag = np.mean(np.abs(up_mag * w * xhat), axis=-1, keepdims=True)
    dx = r * (up * w - xhat * inner)
    dx_bound = gamma(2 * D + 30) * r * (up_mag * np.abs(w) + np.abs(xhat) * inner_mag)
    axes = tuple(range(x.ndim - 1))
    n = x.size // D
    dw = (up * xhat).sum(axes)
    dw_bound = gamma(n + D / 2 + 12) * (up_mag * np.abs(xhat)).sum(axes)
    return dx, dx_bound, dw, dw_bound


# --------------------------------------------------------------------------
# paged append
# --------------------------------------------------------------------------
def append(cache, rows, slots):
    """cache [pages, page_size, heads, dim] with the tokens' rows written."""
    out = np.array(cache)
    pages, page = out.shape[:2]
    for t, s in enumerate(slots):
        if 0 <= s < pages * page:
            out[s // page, s % page] = rows[t]
    return out

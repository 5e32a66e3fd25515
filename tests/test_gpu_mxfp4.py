"""GPU parity of MXFP4 codes, values, products and gradients.

Codes, scales and values are defined bit for bit.  The product sums in fp32 in
an order of its own: with operands whose sums fp32 holds exactly the bar is bit
equality, with others the bound of the oracle."""

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer, mx
from tests.gpu_util import assert_bits_equal, bits, case, dev, torch
from tests.test_gpu_int8 import DT, make, tdt, upload

pytestmark = pytest.mark.gpu

INF = {"fp32": 0x7F800000, "fp16": 0x7C00, "bf16": 0x7F80}
NAN = {"fp32": 0x7FC00001, "fp16": 0x7E01, "bf16": 0x7FC1}


def u8(a, ld=None, fill=0xEE, shift=0):
    """uint8 matrix on the device, rows ld bytes apart, `shift` bytes into its buffer."""
    t = torch()
    rows, d = a.shape
    ld = d if ld is None else ld
    buf = t.full((max(rows, 1) * ld + shift,), fill, dtype=t.uint8, device=dev())
    out = t.as_strided(buf, (rows, d), (ld, 1), shift)
    out.copy_(t.from_numpy(np.ascontiguousarray(a)).to(dev()))
    return out


def same_codes(got, want, what):
    for g, w, name in zip(got, want, ("codes", "scales")):
        assert_bits_equal(g.cpu().numpy(), w, f"{what}: {name}")


# --------------------------------------------------------------------------
# quantize, dequantize
# --------------------------------------------------------------------------
@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 31), (2, 32), (3, 33), (5, 511), (1, 4096), (64, 513), (7, 2049), (130, 96),
                                    (2, 20001)])
def test_rows_and_columns(t, rows, d):
    case(f"mxfp4 quantize {t} {rows}x{d}")
    b, x = make(np.random.default_rng(rows * 7 + d), (rows, d), t)
    want = mx.quantize(x)
    X = upload(b, t)
    got = kb.quantize_mxfp4(X)
    same_codes(got, want, "rows")
    back = kb.dequantize_mxfp4(*got, d, dtype=tdt(t))
    assert_bits_equal(bits(back), layer.round_to(mx.values(*want, d).astype(np.float32), t), "values")
    want_c = mx.quantize(np.ascontiguousarray(x.T))
    if rows > 1 and d > 1:
        assert X.t().stride() == (1, d)
    same_codes(kb.quantize_mxfp4(X.t()), want_c, "columns")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("rows,d,ld,start", [(300, 70, 71, 0), (70, 200, 256, 1), (257, 130, 136, 2), (40, 129, 136, 3)])
def test_strided_inputs_and_given_buffers(t, rows, d, ld, start):
    T = torch()
    case(f"mxfp4 quantize strided {t} {rows}x{d} ld {ld} start {start}")
    b, x = make(np.random.default_rng(rows + d), (rows, ld + 8), t)
    whole = upload(b, t)
    X = T.as_strided(whole, (rows, d), (ld + 8, 1), start)
    x = x[:, start:start + d]
    for v, want in ((X, mx.quantize(x)), (X.t(), mx.quantize(np.ascontiguousarray(x.T)))):
        n, nb = want[1].shape
        codes, scales = u8(np.zeros_like(want[0]), 16 * nb + 32), u8(np.zeros_like(want[1]), nb + 3, shift=1)
        out = kb.quantize_mxfp4(v, codes, scales)
        assert out[0] is codes or out[0].data_ptr() == codes.data_ptr()
        same_codes((codes, scales), want, "given")
        for buf, inner in ((codes, 16 * nb), (scales, nb)):  # what lies between the rows is left alone
            ld_b = buf.stride(0)
            all_rows = T.as_strided(buf, (n - 1, ld_b), (ld_b, 1), buf.storage_offset()).cpu().numpy()
            assert (all_rows[:, inner:] == 0xEE).all()
        out = T.full((n, v.shape[1] + 5), 7.0, dtype=tdt(t), device=dev())
        kb.dequantize_mxfp4(codes, scales, v.shape[1], dtype=tdt(t), out=out[:, 2:2 + v.shape[1]])
        got = out.float().cpu().numpy()
        assert np.array_equal(got[:, 2:-3], mx.values(*want, v.shape[1])) and (got[:, :2] == 7).all() and (got[:, -3:] == 7).all()


@pytest.mark.parametrize("t", ["fp16", "bf16"])
def test_every_value_of_a_type_under_many_scales(t):
    # 31 neighbours of all finite patterns a block, and a driver that sets the scale
    n = INF[t]
    every = np.concatenate([np.arange(n), np.arange(n) + 0x8000]).astype(np.uint16)
    pad = np.zeros(-every.size % 31, np.uint16)
    b = np.concatenate([every, pad]).reshape(-1, 31)
    expo = 10 if t == "fp16" else 7
    for up in (0, 1, 2, 3, 4, 6, 40):
        top = np.minimum((b & 0x7FFF).max(1) + (up << expo), n - 1).astype(np.uint16)
        x = np.ascontiguousarray(np.concatenate([b, top[:, None]], 1).reshape(8, -1))
        case(f"mxfp4 every {t} value, driver {up}")
        got = kb.quantize_mxfp4(upload(x, t))
        same_codes(got, mx.quantize(layer.values(x, t)), f"driver {up}")


@pytest.mark.parametrize("t", DT)
def test_special_blocks(t):
    size = {"fp32": np.uint32, "fp16": np.uint16, "bf16": np.uint16}[t]
    x = np.zeros((9, 100), np.float32)
    x[3] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -5.0], 10)  # ties
    x[4] = -x[3] * 4
    x[5] = 1.0
    b = layer.round_to(x, t).astype(size)
    b[1, 40], b[2, 99], b[5, 7] = INF[t], INF[t] | (1 << (8 * b.itemsize - 1)), NAN[t]
    b[6] = np.arange(1, 101)                     # subnormals
    b[7] = np.arange(1, 101) | (1 << (8 * b.itemsize - 1))
    b[8] = INF[t] - 1 - np.arange(100)           # the largest values
    b[0, 1] = 1 << (8 * b.itemsize - 1)          # -0
    case(f"mxfp4 special {t}")
    X = upload(b, t)
    want = mx.quantize(layer.values(b, t))
    got = kb.quantize_mxfp4(X)
    same_codes(got, want, "rows")
    back = kb.dequantize_mxfp4(*got, 100, dtype=tdt(t)).float().cpu().numpy()
    assert np.array_equal(back, mx.values(*want, 100).astype(np.float32), equal_nan=True)
    same_codes(kb.quantize_mxfp4(X.t()), mx.quantize(np.ascontiguousarray(layer.values(b, t).T)), "columns")


def test_fp32_of_every_exponent():
    rng = np.random.default_rng(8)
    b = np.repeat(np.arange(255, dtype=np.uint32) << 23, 64).reshape(255, 64)
    b = b | rng.integers(0, 1 << 23, b.shape).astype(np.uint32) | rng.integers(0, 2, b.shape).astype(np.uint32) << 31
    for spread in (0, 3, 30):
        x = b.copy()
        x[:, 1:] -= np.minimum(rng.integers(0, spread + 1, (255, 63)).astype(np.uint32), (x[:, 1:] >> 23) & 255) << 23
        case(f"mxfp4 fp32 exponents {spread}")
        got = kb.quantize_mxfp4(upload(x, "fp32"))
        same_codes(got, mx.quantize(x.view(np.float32)), f"spread {spread}")


@pytest.mark.parametrize("t", DT)
def test_values_of_every_code_and_scale(t):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))        # 16 blocks a row
    scales = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 16))
    case(f"mxfp4 values {t}")
    got = kb.dequantize_mxfp4(u8(codes), u8(scales), 512, dtype=tdt(t))
    with np.errstate(over="ignore"):
        want = mx.values(codes, scales).astype(np.float32)
    ok = scales[:, :1].repeat(512, 1) != 255
    assert_bits_equal(np.where(ok, bits(got), 0), np.where(ok, layer.round_to(want, t), 0), "values")
    assert np.isnan(got.float().cpu().numpy()[~ok]).all()


def test_no_rows():
    T = torch()
    for t in DT:
        x = T.empty((0, 70), dtype=tdt(t), device=dev())
        codes, scales = kb.quantize_mxfp4(x)
        assert codes.shape == (0, 48) and scales.shape == (0, 3)
        assert kb.dequantize_mxfp4(codes, scales, 70, dtype=tdt(t)).shape == (0, 70)


# --------------------------------------------------------------------------
# product
# --------------------------------------------------------------------------
def random_codes(rng, rows, d, lo=126, hi=128):
    """Codes and scales as a quantizer leaves them (zeros past d); with scales
    of 2^-1 .. 2^1 sums are multiples of 2^-4 below 36 * 4 d: exact in fp32 up to
    d = 7281."""
    c = rng.integers(0, 16, (rows, mx.blocks(d) * 32)).astype(np.uint8)
    c[:, d:] = 0
    return c[:, 0::2] | c[:, 1::2] << 4, rng.integers(lo, hi + 1, (rows, mx.blocks(d))).astype(np.uint8)


SHAPES = [(1, 1, 1), (1, 4096, 512), (1, 17, 4099), (3, 64, 63), (5, 33, 64), (8, 128, 1000), (16, 256, 256),
          (16, 50, 2048), (17, 130, 192), (31, 65, 129), (33, 96, 320), (64, 64, 64), (65, 257, 100), (77, 300, 1040),
          (128, 128, 128), (129, 255, 384), (200, 511, 80), (256, 256, 512), (257, 513, 272), (300, 1000, 16),
          (512, 768, 640), (1000, 520, 144), (16, 9, 4100), (48, 7000, 500), (112, 4000, 700), (600, 600, 7000)]


def product_case(M, N, K, t, bias=True, seed=0):
    rng = np.random.default_rng(M * 31 + N * 7 + K + seed)
    a, w = random_codes(rng, M, K), random_codes(rng, N, K)
    bb = layer.round_to((rng.integers(-64, 65, N) / 4).astype(np.float32), t) if bias else None
    y = mx.values(*a) @ mx.values(*w).T  # exact
    if bias:
        y = y + layer.values(bb, t)
    return a, w, bb, layer.round_to(y.astype(np.float32), t)


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(t, M, N, K):
    case(f"linear mxfp4 {t} M={M} N={N} K={K}")
    a, w, bb, want = product_case(M, N, K, t, bias=(M + N) % 2 == 0)
    got = kb.linear_mxfp4(u8(a[0]), u8(a[1]), u8(w[0]), u8(w[1]), bias=None if bb is None else upload(bb[None], t)[0],
                          dtype=tdt(t))
    assert_bits_equal(bits(got), want, f"product {M} {N} {K}")


FEW = [(16, 16), (16, 32), (16, 48), (16, 64), (32, 32), (32, 64), (48, 32), (48, 64), (64, 64), (80, 48), (80, 64), (112, 48),
       (128, 48)]


@pytest.mark.parametrize("K", [32, 700, 2048])
def test_product_at_tile_borders(K):
    # rows and channels around every tile's size, a partial and a whole step
    for M in sorted({m for r, _ in FEW for m in (r - 1, r, r + 1)} | {255, 256, 257}):
        N = 100 + M
        a, w, bb, want = product_case(M, N, K, "bf16")
        case(f"linear mxfp4 borders M={M} N={N} K={K}")
        got = kb.linear_mxfp4(u8(a[0]), u8(a[1]), u8(w[0]), u8(w[1]), bias=upload(bb[None], "bf16")[0])
        assert_bits_equal(bits(got), want, f"product {M} {N} {K}")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", [(4096, 4096, 512), (2100, 5000, 1000), (5000, 2111, 768), (4100, 4104, 1030), (8192, 1024, 256)])
def test_product_of_many_tiles(t, M, N, K):
    case(f"linear mxfp4 large {t} M={M} N={N} K={K}")
    a, w, bb, want = product_case(M, N, K, t)
    got = kb.linear_mxfp4(u8(a[0]), u8(a[1]), u8(w[0]), u8(w[1]), bias=upload(bb[None], t)[0], dtype=tdt(t))
    assert_bits_equal(bits(got), want, f"product {M} {N} {K}")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", [(5, 70, 300), (1, 64, 96), (70, 33, 1000), (300, 300, 544), (130, 1100, 2000)])
def test_product_strides(t, M, N, K):
    # rows of codes 16-byte multiples apart, of scales at any byte, an output
    # inside a larger one
    T = torch()
    a, w, bb, want = product_case(M, N, K, t)
    ka, kc = a[0].shape[1], a[1].shape[1]
    for pa, pw, sa, sw, lo in ((16, 0, 1, 2, 3), (0, 48, 3, 0, 8), (256, 16, 5, 7, 1)):
        case(f"linear mxfp4 strides {t} M={M} N={N} K={K} {pa} {pw} {sa} {sw} {lo}")
        out = T.full((M, N + 16), 9.0, dtype=tdt(t), device=dev())
        kb.linear_mxfp4(u8(a[0], ka + pa), u8(a[1], kc + sa, 0xFF, sa), u8(w[0], ka + pw), u8(w[1], kc + sw, 0xFF, sw),
                        bias=upload(bb[None], t)[0], dtype=tdt(t), out=out[:, lo:lo + N])
        assert_bits_equal(bits(out[:, lo:lo + N].contiguous()), want, "product")
        assert (out[:, :lo] == 9).all() and (out[:, lo + N:] == 9).all()


@pytest.mark.parametrize("M,N,K", [(3, 40, 600), (70, 90, 1100), (400, 300, 2085), (1100, 2000, 512)])
def test_product_of_far_scales(M, N, K):
    # scales over the whole range of activations and weights: the oracle's bound
    rng = np.random.default_rng(M)
    a, w = random_codes(rng, M, K, 100, 150), random_codes(rng, N, K, 90, 130)
    case(f"linear mxfp4 far scales M={M} N={N} K={K}")
    y, bound = mx.product(mx.values(*a), mx.values(*w))
    got = kb.linear_mxfp4(u8(a[0]), u8(a[1]), u8(w[0]), u8(w[1]), dtype=torch().float32).cpu().numpy()
    assert (np.abs(got - y) <= bound).all(), float((np.abs(got - y) / bound).max())


@pytest.mark.parametrize("M,N,K", [(1, 64, 128), (6, 40, 600), (100, 90, 1100), (300, 300, 2085), (1024, 1024, 512)])
def test_product_of_the_ends_of_the_scales(M, N, K):
    # one block a row counts, in the other all scales are the least or the largest: 2^-127 2^127
    rng = np.random.default_rng(M + 1)
    for lo, hi in ((0, 254), (254, 0)):
        a, w = random_codes(rng, M, K, lo, lo), random_codes(rng, N, K, hi, hi)
        case(f"linear mxfp4 ends of the scales M={M} N={N} K={K} {lo}")
        y = mx.values(*a) @ mx.values(*w).T
        got = kb.linear_mxfp4(u8(a[0]), u8(a[1]), u8(w[0]), u8(w[1]), dtype=torch().float32)
        assert_bits_equal(bits(got), y.astype(np.float32).view(np.uint32), "product")


@pytest.mark.parametrize("M,N,K", [(1, 40, 600), (5, 40, 600), (70, 90, 1100), (300, 300, 2085), (2500, 2304, 512)])
def test_product_of_blocks_that_are_nan(M, N, K):
    a, w, _, _ = product_case(M, N, K, "fp32", bias=False)
    y = mx.values(*a) @ mx.values(*w).T
    nb = mx.blocks(K)
    rng = np.random.default_rng(5)
    rows, chans = rng.choice(M, max(1, M // 7), replace=False), rng.choice(N, max(1, N // 9), replace=False)
    if M == 1:
        rows = rows[:0]
    for r in rows:
        b = int(rng.integers(0, nb))
        a[1][r, b] = 255
        a[0][r, 16 * b:16 * b + 16] = 0
    for c in chans:
        b = int(rng.integers(0, nb))
        w[1][c, b] = 255
        w[0][c, 16 * b:16 * b + 16] = 0
    case(f"linear mxfp4 NaN blocks M={M} N={N} K={K}")
    got = kb.linear_mxfp4(u8(a[0]), u8(a[1]), u8(w[0]), u8(w[1]), dtype=torch().float32).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[rows] = True
    want[:, chans] = True
    assert np.array_equal(np.isnan(got), want)
    assert np.array_equal(got[~want], y[~want].astype(np.float32))


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", [(1, 4096, 512), (1, 17, 4099), (1, 100, 1), (2, 1, 130), (3, 64, 63), (4, 700, 2049), (8, 128, 1000),
                                   (8, 5000, 255), (7, 14336, 96), (1, 12300, 3000), (9, 65, 129), (33, 96, 320), (300, 511, 777)])
def test_dynamic(t, M, N, K):
    rng = np.random.default_rng(M + N + K)
    # values on a grid, so that all sums are exact: codes of every block have the scale 2^0 to 2^1
    x = rng.choice([0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -2, -3, -5, 7, 12], (M, K)).astype(np.float32)
    w = random_codes(rng, N, K)
    bb = layer.round_to((rng.integers(-64, 65, N) / 4).astype(np.float32), t)
    want = mx.rounded(x) @ mx.values(*w)[:, :K].T + layer.values(bb, t)
    case(f"linear mxfp4 dynamic {t} M={M} N={N} K={K}")
    for lead in (0, 1):  # rows of X that start at 16 bytes, and not
        X = torch().zeros((M, K + 8 + lead), dtype=tdt(t), device=dev())[:, lead:lead + K]
        X.copy_(torch().from_numpy(x).to(dev()))
        got = kb.linear_mxfp4_dynamic(X, u8(w[0]), u8(w[1], w[1].shape[1] + 1), bias=upload(bb[None], t)[0])
        assert_bits_equal(bits(got), layer.round_to(want.astype(np.float32), t), f"dynamic, lead {lead}")


@pytest.mark.parametrize("M", [1, 4, 9, 200])
def test_dynamic_of_tokens_that_are_not_finite(M):
    T = torch()
    rng = np.random.default_rng(M)
    K, N = 700, 90
    b, x = make(rng, (M, K), "bf16")
    w = random_codes(rng, N, K)
    b[M // 2, 650] = NAN["bf16"]
    b[0, 3] = INF["bf16"]
    case(f"linear mxfp4 dynamic of NaN M={M}")
    got = kb.linear_mxfp4_dynamic(upload(b, "bf16"), u8(w[0]), u8(w[1])).float().cpu().numpy()
    bad = np.zeros(M, bool)
    bad[[0, M // 2]] = True
    assert np.isnan(got[bad]).all() and np.isfinite(got[~bad]).all()
    assert kb.linear_mxfp4_dynamic(T.empty((0, K), dtype=T.bfloat16, device=dev()), u8(w[0]), u8(w[1])).shape == (0, N)


def test_a_weight_of_one_channel_and_rows_past_the_last():
    rng = np.random.default_rng(1)
    for M in (1, 6, 40, 300):
        a, w = random_codes(rng, M, 96), random_codes(rng, 1, 96)
        case(f"linear mxfp4 one channel M={M}")
        got = kb.linear_mxfp4(u8(a[0]), u8(a[1]), u8(w[0]), u8(w[1]), dtype=torch().float32).cpu().numpy()
        assert np.array_equal(got, mx.values(*a) @ mx.values(*w).T)


# --------------------------------------------------------------------------
# gradients
# --------------------------------------------------------------------------
def within(got, want, bound, t, what):
    rel, least = layer.half_ulp(t)
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    limit = bound + rel * (np.abs(want) + bound) + least
    bad = ~(err <= limit)
    assert not bad.any(), (what, int(bad.sum()), float((err / np.maximum(limit, 1e-300)).max()))


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 96), (7, 33, 65), (32, 32, 32), (100, 70, 300), (257, 130, 191), (300, 513, 1000),
                                   (1000, 520, 257)])
def test_backward(t, M, N, K):
    T = torch()
    rng = np.random.default_rng(M + 3 * N + K)
    gb, g = make(rng, (M, N), t)
    xb, x = make(rng, (M, K), t)
    wb, w = make(rng, (N, K), t, 0.5)
    G, X, W = upload(gb, t), upload(xb, t), upload(wb, t)
    case(f"linear mxfp4 backward {t} M={M} N={N} K={K}")
    (dx, ex), (dw, ew), (db, eb) = mx.linear_backward(g, x, w)
    got = kb.linear_mxfp4_backward(G, X, W)
    assert got[0].dtype == tdt(t) and got[1].dtype == got[2].dtype == T.float32
    within(got[0], dx, ex, t, "dx")
    within(got[1], dw, ew, "fp32", "dw")
    within(got[2], db, eb, "fp32", "db")
    # each alone gives the same bits, into a given output as well
    for i, only in enumerate(((True, False, False), (False, True, False), (False, False, True))):
        alone = kb.linear_mxfp4_backward(G, X, W, *only)
        assert [v is not None for v in alone] == list(only)
        assert_bits_equal(bits(alone[i]), bits(got[i]), f"alone {i}")
    out = T.full((M, K + 9), 5.0, dtype=tdt(t), device=dev())
    out_w = T.full((N, K + 3), 5.0, dtype=T.float32, device=dev())
    kb.linear_mxfp4_backward(G, X, W, dX=out[:, 1:K + 1], dweight=out_w[:, 2:K + 2])
    assert_bits_equal(bits(out[:, 1:K + 1].contiguous()), bits(got[0]), "dX in a larger one")
    assert_bits_equal(bits(out_w[:, 2:K + 2].contiguous()), bits(got[1]), "dweight in a larger one")
    assert (out[:, :1] == 5).all() and (out[:, K + 1:] == 5).all() and (out_w[:, :2] == 5).all() and (out_w[:, K + 2:] == 5).all()


def test_backward_without_tokens():
    T = torch()
    g, x, w = (T.ones(s, device=dev(), dtype=T.bfloat16) for s in ((0, 40), (0, 50), (40, 50)))
    case("linear mxfp4 backward of no tokens")
    dx, dw, db = kb.linear_mxfp4_backward(g, x, w, dweight=T.full((40, 50), 3.0, device=dev()))
    assert dx.shape == (0, 50) and (dw == 0).all() and (db == 0).all()


def test_backward_of_values_that_are_not_finite():
    # a NaN of dout reaches its row of dX and its channel of dW and db
    T = torch()
    M, N, K = 70, 40, 50
    g, x, w = T.ones((M, N), device=dev()), T.ones((M, K), device=dev()), T.ones((N, K), device=dev())
    g[20, 7] = float("nan")
    case("linear mxfp4 backward of NaN")
    dx, dw, db = (v.cpu().numpy() for v in kb.linear_mxfp4_backward(g, x, w))
    want = np.zeros((M, K), bool)
    want[20] = True
    assert np.array_equal(np.isnan(dx), want)
    want = np.zeros((N, K), bool)
    want[7] = True
    assert np.array_equal(np.isnan(dw), want) and np.isnan(db).tolist() == [i == 7 for i in range(N)]


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_large_products_of_odd_depth_in_used_workspaces(t):
    # depths that end inside a pair of steps, in workspaces full of NaN scales
    T = torch()
    M, N, K = 4100, 1030, 4104
    rng = np.random.default_rng(9)
    grid = np.array([0.5, 1, 1.5, 2, 3, 4, 6, -0.5, -1, -2, -3], np.float32)
    g, w = (rng.choice(grid, s).astype(np.float32) for s in ((M, N), (N, K)))
    G, W = (T.from_numpy(v).to(dev()).to(tdt(t)) for v in (g, w))
    lib = kb.lib()

    def used(n):
        return T.full((n,), 0xFF, dtype=T.uint8, device=dev())
    case(f"large dynamic product of odd depth {t}")
    wt = mx.quantize(np.ascontiguousarray(w.T))
    want = layer.round_to((mx.rounded(g) @ mx.values(*wt, N).T).astype(np.float32), t)
    got = kb.linear_mxfp4_dynamic(G, u8(wt[0]), u8(wt[1]), workspace=used(lib.linear_mxfp4_dynamic_workspace_bytes(M, K, N)))
    assert_bits_equal(bits(got), want, "dynamic")
    case(f"large product of codes of odd depth {t}")
    gq = mx.quantize(g)
    got = kb.linear_mxfp4(u8(gq[0]), u8(gq[1]), u8(wt[0]), u8(wt[1]), dtype=tdt(t),
                          workspace=used(lib.linear_mxfp4_workspace_bytes(M, K, 32 * wt[1].shape[1])))
    assert_bits_equal(bits(got), want, "codes")
    case(f"large gradients of odd depth {t}")
    x = rng.choice(grid, (M, K)).astype(np.float32)
    dx, dw, db = kb.linear_mxfp4_backward(G, T.from_numpy(x).to(dev()).to(tdt(t)), W,
                                          workspace=used(lib.linear_mxfp4_backward_workspace_bytes(M, N, K)))
    assert_bits_equal(bits(dx), want, "dX")
    want = mx.rounded(np.ascontiguousarray(g.T)) @ mx.rounded(np.ascontiguousarray(x.T)).T
    assert_bits_equal(bits(dw), want.astype(np.float32).view(np.uint32), "dW")
    assert np.array_equal(db.cpu().numpy(), g.sum(0))

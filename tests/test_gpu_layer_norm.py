"""GPU parity of the layer norm and its gradients: float64 values with the
oracle's bound of an fp32 evaluation, then one rounding to the type."""

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer, mx
from tests.gpu_util import assert_bits_equal, bits, case, dev, torch
from tests.test_gpu_int8 import DT, make, tdt, upload
from tests.test_gpu_mxfp4 import INF, NAN, within

pytestmark = pytest.mark.gpu

# around every form's longest row, odd ones and those that start at 16 bytes
SIZES = [(1, 1), (5, 2), (3, 7), (9, 64), (4, 511), (5, 512), (6, 513), (3, 1024), (1100, 1000), (1030, 777), (3, 2047), (5, 2048),
         (2, 2056), (7, 4096), (3, 4097), (2, 8192), (3, 8193), (2, 8200), (3, 16384), (2, 16392), (2, 32768), (2, 32769),
         (2, 40000), (1, 70000), (2, 65543), (515, 24), (700, 1025), (2100, 40), (1, 4096), (513, 2048)]


def data(t, rows, d, seed=0, shift=1.0):
    rng = np.random.default_rng(rows * 13 + d + seed)
    b, x = make(rng, (rows, d), t)
    x = x + shift * rng.standard_normal((rows, 1)).astype(np.float32)  # rows whose mean is not zero
    b = layer.round_to(x, t)
    w = layer.round_to((1 + 0.2 * rng.standard_normal(d)).astype(np.float32), t)
    bias = layer.round_to(rng.standard_normal(d).astype(np.float32), t)
    gb, g = make(rng, (rows, d), t, 0.5)
    return b, layer.values(b, t), w, layer.values(w, t), bias, layer.values(bias, t), gb, g


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("rows,d", SIZES)
def test_forward_and_backward(t, rows, d):
    case(f"layer norm {t} {rows}x{d}")
    b, x, wb, w, bb, bias, gb, g = data(t, rows, d)
    X, W, B, G = upload(b, t), upload(wb[None], t)[0], upload(bb[None], t)[0], upload(gb, t)
    y = kb.layer_norm(X, W, B)
    within(y, *mx.layer_norm(x, w, bias, 1e-5), t, "forward")
    within(kb.layer_norm(X, W, eps=0.1), *mx.layer_norm(x, w, None, 0.1), t, "without bias")
    (dx, ex), (dw, ew), (db, eb) = mx.layer_norm_back(g, x, w, 1e-5)
    got = kb.layer_norm_backward(G, X, W)
    assert got[0].dtype == tdt(t) and got[1].dtype == got[2].dtype == torch().float32
    within(got[0], dx, ex, t, "dx")
    within(got[1], dw, ew, "fp32", "dw")
    within(got[2], db, eb, "fp32", "db")
    again = kb.layer_norm_backward(G, X, W)
    for a, c, name in zip(got, again, ("dx", "dw", "db")):
        assert_bits_equal(bits(a), bits(c), f"a second run: {name}")
    # in place
    assert_bits_equal(bits(kb.layer_norm(X.clone(), W, B, out=None)), bits(y), "again")
    X2, G2 = X.clone(), G.clone()
    kb.layer_norm_backward(G2, X2, W, dx=G2)
    assert_bits_equal(bits(G2), bits(got[0]), "dx over dout")
    kb.layer_norm(X2, W, B, out=X2)
    assert_bits_equal(bits(X2), bits(y), "out over x")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("rows,d", [(5, 2), (9, 64), (600, 777), (1030, 3000), (600, 8000), (600, 9001), (600, 16392), (3, 70001)])
def test_gradients_over_dout(t, rows, d):
    # the weights' gradients come from dout as it was
    T = torch()
    case(f"layer norm gradients over dout {t} {rows}x{d}")
    b, x, wb, w, bb, bias, gb, g = data(t, rows, d, 3)
    X, W = upload(b, t), upload(wb[None], t)[0]
    want = kb.layer_norm_backward(upload(gb, t), X, W)
    wide = T.full((rows, d + 3), 2.0, dtype=tdt(t), device=dev())
    for G in (upload(gb, t), wide[:, 1:d + 1]):
        G.copy_(upload(gb, t))
        got = kb.layer_norm_backward(G, X, W, dx=G)
        for a, c, name in zip((G.contiguous(), *got[1:]), want, ("dx", "dweight", "dbias")):
            assert_bits_equal(bits(a), bits(c), name)
    assert (wide[:, 0] == 2).all() and (wide[:, d + 1:] == 2).all()


@pytest.mark.parametrize("t", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,d", [(3, 100), (40, 512), (70, 3000), (3, 12000), (2, 20000), (2, 70001)])
def test_weights_in_fp32(t, rows, d):
    T = torch()
    case(f"layer norm {t} {rows}x{d}, fp32 weights")
    b, x, _, _, _, _, gb, g = data(t, rows, d, 1)
    rng = np.random.default_rng(d)
    w, bias = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32), rng.standard_normal(d).astype(np.float32)
    W, B = T.from_numpy(w).to(dev()), T.from_numpy(bias).to(dev())
    within(kb.layer_norm(upload(b, t), W, B), *mx.layer_norm(x, w, bias, 1e-5), t, "forward")
    want = mx.layer_norm_back(g, x, w, 1e-5)
    for got, (v, e), ty in zip(kb.layer_norm_backward(upload(gb, t), upload(b, t), W), want, (t, "fp32", "fp32")):
        within(got, v, e, ty, "gradient")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("rows,d,ld,start", [(7, 64, 72, 8), (7, 64, 71, 3), (5, 700, 1000, 1), (3, 5000, 5008, 0), (3, 9000, 9002, 1),
                                             (2, 16000, 16008, 1), (2, 33000, 33000, 0)])
def test_strided_rows(t, rows, d, ld, start):
    T = torch()
    case(f"layer norm strided {t} {rows}x{d} ld {ld} start {start}")
    b, x, wb, w, bb, bias, gb, g = data(t, rows, d, 2)

    def strided(v):
        buf = T.full((rows * ld + start,), 3.0, dtype=tdt(t), device=dev())
        s = T.as_strided(buf, (rows, d), (ld, 1), start)
        if v is not None:
            s.copy_(upload(v, t))
        return buf, s
    W, B = upload(wb[None], t)[0], upload(bb[None], t)[0]
    _, X = strided(b)
    _, G = strided(gb)
    for out, run, checks in (
            (strided(None), lambda o: [kb.layer_norm(X, W, B, out=o)], [mx.layer_norm(x, w, bias, 1e-5)]),
            (strided(None), lambda o: kb.layer_norm_backward(G, X, W, dx=o), mx.layer_norm_back(g, x, w, 1e-5))):
        got = run(out[1])
        for i, (v, e) in enumerate(checks):
            within(got[i], v, e, t if i == 0 else "fp32", f"output {i}")
        rest = T.ones(rows * ld + start, dtype=T.bool, device=dev())
        T.as_strided(rest, (rows, d), (ld, 1), start).fill_(False)
        assert (out[0][rest] == 3.0).all()


@pytest.mark.parametrize("d", [5, 64, 700, 2048, 5000, 9000, 20000, 40000, 70000])
def test_rows_far_from_zero(d):
    # a mean 3000 times the deviation: fp32 sums of x alone would lose the row
    case(f"layer norm far from zero {d}")
    for offset in (1000.0, -30000.0):
        rng = np.random.default_rng(d)
        x = (offset + rng.standard_normal((3, d)) * abs(offset) / 3000).astype(np.float32)
        g = rng.standard_normal((3, d)).astype(np.float32)
        w = np.ones(d, np.float32)
        X, G, W = upload(x.view(np.uint32), "fp32"), upload(g.view(np.uint32), "fp32"), upload(w[None].view(np.uint32), "fp32")[0]
        y, _ = mx.layer_norm(x, w, None, 1e-5)
        got = kb.layer_norm(X, W).double().cpu().numpy()
        # x - m0 is off by u |x - m0| at most where x is within a factor of two of m0 (it is exact), m1 by
        # g(depth) of mean|x - m0|, and |x - m0| <= |c| + |m1| with |m1| <= g(depth) |mean|: 2^-24 * 100 * 3000 deviations
        D = 96 + d // 1024
        limit = layer.gamma(D + 8) * (np.abs(y) + 1) * (1 + np.abs(y)) * (1 + layer.gamma(D) * 6000)
        assert (np.abs(got - y) <= limit).all(), float((np.abs(got - y) / limit).max())
        dx, dw, db = (v.double().cpu().numpy() for v in kb.layer_norm_backward(G, X, W))
        for got, (v, e) in zip((dx, dw, db), mx.layer_norm_back(g, x, w, 1e-5)):
            assert (np.abs(got - v) <= e + 2.0 ** -24 * np.abs(v)).all()


@pytest.mark.parametrize("d", [1, 40, 600, 3000, 9000, 17000, 33000, 70000])
def test_special_rows(d):
    # constant rows, zeros, a NaN, an infinity: each stays in its row (dx) and, for finite rows, gives the formula's values
    T = torch()
    case(f"layer norm special {d}")
    x = np.tile(np.linspace(-1, 1, d).astype(np.float32), (6, 1))
    x[0], x[1] = 3.25, 0.0
    x[2, d // 2], x[3, d - 1] = np.nan, np.inf
    rng = np.random.default_rng(d)
    g = rng.standard_normal((6, d)).astype(np.float32)
    w, bias = rng.standard_normal(d).astype(np.float32), rng.standard_normal(d).astype(np.float32)
    X, G, W, B = (T.from_numpy(v).to(dev()) for v in (x, g, w, bias))
    got = kb.layer_norm(X, W, B).cpu().numpy()
    assert np.array_equal(got[0], bias) and np.array_equal(got[1], bias)
    assert np.isnan(got[2:4]).all() and np.isfinite(got[4:]).all()
    dx, dw, db = (v.cpu().numpy() for v in kb.layer_norm_backward(G, X, W))
    assert np.isnan(dx[2:4]).all() and np.isfinite(dx[[0, 1, 4, 5]]).all() and np.isnan(dw).all()
    assert np.isfinite(db).all()
    keep = [0, 1, 4, 5]
    for got, (v, e) in zip(kb.layer_norm_backward(G[keep], X[keep], W), mx.layer_norm_back(g[keep], x[keep], w, 1e-5)):
        within(got, v, e, "fp32", "finite rows")


def test_no_rows():
    T = torch()
    for d in (40, 5000, 20000):
        x, w = T.empty((0, d), device=dev()), T.ones(d, device=dev())
        case(f"layer norm of no rows {d}")
        assert kb.layer_norm(x, w).shape == (0, d)
        dx, dw, db = kb.layer_norm_backward(x, x, w)
        assert dx.shape == (0, d) and (dw == 0).all() and (db == 0).all()


def test_not_finite_16_bit():
    for t in ("fp16", "bf16"):
        b, x, wb, w, *_ = data(t, 4, 300)
        b[1, 7], b[2, 299] = NAN[t], INF[t]
        case(f"layer norm {t} not finite")
        got = kb.layer_norm(upload(b, t), upload(wb[None], t)[0]).float().cpu().numpy()
        assert np.isnan(got[1:3]).all() and np.isfinite(got[[0, 3]]).all()

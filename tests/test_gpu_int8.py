"""GPU parity of the int8 rows and their product.

Every rounding of both is defined and the sums are integers, so the bar is
bit equality with the oracle, at every size and alignment."""

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer
from tests.gpu_util import TORCH_DT, assert_bits_equal, assert_f32_bits_equal_nan_as_nan, bits, case, dev, to_dev, torch

pytestmark = pytest.mark.gpu

DT = ["fp32", "fp16", "bf16"]


def tdt(t):
    return getattr(torch(), TORCH_DT[t])


def make(rng, shape, t, spread=2.0):
    """(raw bits, fp32 values) of rows of different magnitude."""
    x = rng.standard_normal(shape) * np.exp(rng.uniform(-spread, spread, (shape[0], 1)))
    b = layer.round_to(x.astype(np.float32), t)
    return b, layer.values(b, t)


def upload(b, t):
    d = torch().from_numpy(np.ascontiguousarray(b).view({2: np.int16, 4: np.int32}[b.dtype.itemsize])).to(dev())
    return d.view(tdt(t)).reshape(b.shape)


def codes_dev(a, pitch=None):
    """int8 matrix with the given row stride (default: 16-byte multiples)."""
    rows, d = a.shape
    pitch = -(-d // 16) * 16 if pitch is None else pitch
    buf = torch().full((max(rows, 1), pitch), 77, dtype=torch().int8, device=dev())[:rows, :d]
    buf.copy_(torch().from_numpy(a).to(dev()))
    return buf


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 4096), (3, 15), (5, 16), (7, 100), (2, 3840), (64, 513), (33, 8191),
                                    (4, 8192), (3, 8200), (2, 20001), (300, 64)])
def test_rows(t, rows, d):
    case(f"int8 rows {t} {rows}x{d}")
    b, x = make(np.random.default_rng(rows * 7 + d), (rows, d), t)
    codes, scale = kb.quantize_rows_int8(upload(b, t))
    q, s = layer.quantize_rows(x)
    assert codes.stride(0) % 16 == 0 or rows == 1
    assert np.array_equal(codes.cpu().numpy(), q)
    assert_bits_equal(bits(scale), s.view(np.uint32), "scale")
    # the padding up to the next multiple of 16 is zero
    pitch = -(-d // 16) * 16
    whole = torch().as_strided(codes, (rows, pitch), (pitch, 1)).cpu().numpy()
    assert not whole[:, d:].any()


@pytest.mark.parametrize("t", DT)
def test_rows_special(t):
    x = np.zeros((8, 200), np.float32)
    x[1, 150] = np.inf
    x[2, 3] = np.nan
    x[3, 199] = -np.inf
    x[4] = np.linspace(-1, 1, 200)
    x[5] = 2.0 ** -101 if t == "bf16" or t == "fp32" else 2.0 ** -24
    x[6, 7] = -65504.0
    x[7] = np.tile([1.0, -0.5, 0.5 / 127, -1.5 / 127], 50)  # ties between codes up to rounding
    b = layer.round_to(x, t)
    b[2, 3] = {"fp32": 0x7FC00000, "fp16": 0x7E00, "bf16": 0x7FC0}[t]
    b[1, 150] = {"fp32": 0x7F800000, "fp16": 0x7C00, "bf16": 0x7F80}[t]
    b[3, 199] = {"fp32": 0xFF800000, "fp16": 0xFC00, "bf16": 0xFF80}[t]
    case(f"int8 rows special {t}")
    codes, scale = kb.quantize_rows_int8(upload(b, t))
    q, s = layer.quantize_rows(layer.values(b, t))
    assert np.array_equal(codes.cpu().numpy(), q)
    assert_f32_bits_equal_nan_as_nan(bits(scale), s.view(np.uint32), "scale")


@pytest.mark.parametrize("t", DT)
def test_rows_strided_and_into_given_buffers(t):
    rng = np.random.default_rng(5)
    b, x = make(rng, (6, 90), t)
    whole = upload(b, t)
    codes = torch().full((6, 160), 55, dtype=torch().int8, device=dev())
    scale = torch().full((8,), 5.0, dtype=torch().float32, device=dev())
    for lo, hi in ((0, 90), (1, 80), (3, 70), (8, 72)):  # every alignment of the first element
        case(f"int8 rows strided {t} {lo}:{hi}")
        codes.fill_(55)
        kb.quantize_rows_int8(whole[:, lo:hi], codes=codes[:, :hi - lo], scale=scale)
        q, s = layer.quantize_rows(x[:, lo:hi])
        got = codes.cpu().numpy()
        assert np.array_equal(got[:, :hi - lo], q)
        end = -(-(hi - lo) // 16) * 16
        assert not got[:, hi - lo:end].any() and (got[:, end:] == 55).all()
        assert_bits_equal(bits(scale)[:6], s.view(np.uint32), "scale")
        assert (scale[6:] == 5.0).all()


SHAPES = [(1, 1, 1), (1, 4096, 512), (1, 17, 4099), (3, 64, 63), (5, 33, 64), (8, 128, 1000), (16, 256, 256),
          (16, 50, 2048), (17, 130, 192), (31, 65, 129), (33, 96, 320), (64, 64, 64), (65, 257, 100), (77, 300, 1040),
          (128, 128, 128), (129, 255, 384), (200, 511, 80), (256, 256, 512), (257, 513, 272), (300, 1000, 16),
          (512, 768, 640), (1000, 520, 144)]


def product_case(M, N, K, t, seed=0, pitches=(None, None), bias=True, low=-128):
    rng = np.random.default_rng(M * 31 + N * 7 + K + seed)
    a = rng.integers(low, 128, (M, K)).astype(np.int8)
    w = rng.integers(low, 128, (N, K)).astype(np.int8)
    sa = rng.uniform(1e-4, 1e-2, M).astype(np.float32)
    sw = rng.uniform(1e-3, 1e-2, N).astype(np.float32)
    bb = layer.round_to(rng.standard_normal(N).astype(np.float32), t) if bias else None
    want = layer.round_to(layer.product(a, sa, w, sw, None if bb is None else layer.values(bb, t)), t)
    got = kb.linear_int8(codes_dev(a, pitches[0]), to_dev(sa), codes_dev(w, pitches[1]), to_dev(sw),
                         bias=None if bb is None else upload(bb[None], t)[0], dtype=tdt(t))
    return got, want


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(t, M, N, K):
    case(f"linear int8 {t} M={M} N={N} K={K}")
    got, want = product_case(M, N, K, t, bias=(M + N) % 2 == 0)
    assert_bits_equal(bits(got), want, f"product {M} {N} {K}")


@pytest.mark.parametrize("M,N,K,px,pw", [(5, 33, 100, 100, 100), (40, 70, 131, 131, 144), (3, 20, 64, 65, 80),
                                         (130, 140, 96, 112, 97), (64, 64, 256, 256, 260)])
def test_product_any_alignment(M, N, K, px, pw):
    case(f"linear int8 unaligned M={M} N={N} K={K} strides {px} {pw}")
    got, want = product_case(M, N, K, "fp32", pitches=(px, pw))
    assert_bits_equal(bits(got), want, "unaligned")


@pytest.mark.parametrize("M", [1, 16, 130, 520])
def test_product_reads_nothing_beyond_the_rows(M):
    # the bytes between K and the row stride hold 77: they must not be summed
    for K in (1, 15, 17, 127, 129, 250):
        case(f"linear int8 tail M={M} K={K}")
        got, want = product_case(M, 270, K, "fp32", pitches=(512, 272))
        assert_bits_equal(bits(got), want, f"K={K}")


@pytest.mark.parametrize("M", [1, 40, 256])
def test_largest_sums(M):
    # K and codes at the limit: the sum reaches 131071 * 2^14, just inside int32
    N, K = 32, 131071
    a = np.full((M, K), -128, np.int8)
    w = np.full((N, K), -128, np.int8)
    w[1::2] = 127
    one = np.ones(max(M, N), np.float32)
    case(f"linear int8 largest sums M={M}")
    got = kb.linear_int8(codes_dev(a), to_dev(one[:M]), codes_dev(w), to_dev(one[:N]), dtype=torch().float32)
    want = np.where(np.arange(N) % 2 == 0, np.float32(131071 * 2 ** 14), np.float32(-131071 * 128 * 127))
    assert np.array_equal(got.cpu().numpy(), np.broadcast_to(want, (M, N)).astype(np.float32))


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", [(1, 256, 4096), (1, 31, 1), (2, 64, 20000), (4, 1000, 250), (16, 128, 4096),
                                   (16, 48, 9000), (17, 64, 512), (100, 200, 300), (300, 300, 1024)])
def test_dynamic_equals_rows_then_product(t, M, N, K):
    case(f"linear int8 dynamic {t} M={M} N={N} K={K}")
    rng = np.random.default_rng(M + N + K)
    b, x = make(rng, (M, K), t)
    if M > 3:
        b[3] = 0
        b[2, K // 2] = {"fp32": 0x7FC00000, "fp16": 0x7E00, "bf16": 0x7FC0}[t]
        x = layer.values(b, t)
    w = rng.integers(-127, 128, (N, K)).astype(np.int8)
    sw = rng.uniform(1e-3, 1e-2, N).astype(np.float32)
    bias = layer.round_to(rng.standard_normal(N).astype(np.float32), t)
    q, s = layer.quantize_rows(x)
    v = layer.product(q, s, w, sw, layer.values(bias, t))
    got = kb.linear_int8_dynamic(upload(b, t), codes_dev(w), to_dev(sw), bias=upload(bias[None], t)[0])
    nan = np.isnan(v)
    assert np.array_equal(torch().isnan(got).cpu().numpy(), nan)
    want = layer.round_to(np.where(nan, 0, v), t)
    assert_bits_equal(np.where(nan, 0, bits(got)), want, "dynamic")


def test_outputs_between_the_rows_stay():
    M, N, K = 37, 50, 96
    rng = np.random.default_rng(8)
    a, w = (rng.integers(-127, 128, s).astype(np.int8) for s in ((M, K), (N, K)))
    sa, sw = (rng.uniform(0.1, 1, n).astype(np.float32) for n in (M, N))
    out = torch().full((M, 64), 3.0, dtype=torch().float32, device=dev())
    case("linear int8 strided out")
    kb.linear_int8(codes_dev(a), to_dev(sa), codes_dev(w), to_dev(sw), dtype=torch().float32, out=out[:, 5:55])
    assert_bits_equal(bits(out[:, 5:55].contiguous()), layer.product(a, sa, w, sw).view(np.uint32), "out")
    assert (out[:, :5] == 3.0).all() and (out[:, 55:] == 3.0).all()


def test_no_rows_and_refusals():
    t = torch()
    w, sw = codes_dev(np.ones((4, 32), np.int8)), t.ones(4, device=dev())
    assert kb.linear_int8(codes_dev(np.ones((0, 32), np.int8)), t.ones(0, device=dev()), w, sw).shape == (0, 4)
    assert kb.linear_int8_dynamic(t.ones(0, 32, device=dev()), w, sw).shape == (0, 4)
    x, sx = codes_dev(np.ones((2, 32), np.int8)), t.ones(2, device=dev())
    for args, kw, match in (((x[:, :31], sx, w, sw), {}, "rows of"), ((x, sx[:1], w, sw), {}, "scale"),
                            ((x, sx, w, sw[:3]), {}, "w_scale"), ((x, sx, w.float(), sw), {}, "w_codes"),
                            ((x, sx, w, sw), {"bias": t.ones(4, device=dev())}, "bias"),
                            ((x, sx, w, sw), {"out": t.ones(2, 4, device=dev())}, "out"),
                            ((x.t(), sx, w, sw), {}, "contiguous"), ((x, sx.cpu(), w, sw), {}, "scale")):
        with pytest.raises((ValueError, TypeError), match=match):
            kb.linear_int8(*args, **kw)
    with pytest.raises(ValueError, match="room"):
        kb.quantize_rows_int8(t.ones(2, 20, device=dev()), codes=t.empty(40, dtype=t.int8, device=dev()).view(2, 20))


def test_on_another_stream_and_in_a_graph():
    t = torch()
    rng = np.random.default_rng(9)
    b, x = make(rng, (24, 640), "bf16")
    w = rng.integers(-127, 128, (96, 640)).astype(np.int8)
    sw = rng.uniform(1e-3, 1e-2, 96).astype(np.float32)
    q, s = layer.quantize_rows(x)
    want = layer.round_to(layer.product(q, s, w, sw), "bf16")
    X, W, S = upload(b, "bf16"), codes_dev(w), to_dev(sw)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    case("linear int8 side stream")
    with t.cuda.stream(side):
        got = kb.linear_int8_dynamic(X, W, S)
    side.synchronize()
    assert_bits_equal(bits(got), want, "side stream")
    case("linear int8 graph")
    out = t.empty_like(got)
    ws = t.empty(kb.lib().linear_int8_dynamic_workspace_bytes(24, 96, 640), dtype=t.uint8, device=dev())
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        kb.linear_int8_dynamic(X, W, S, out=out, workspace=ws)
    for i in range(4):
        out.fill_(0)
        X.copy_(X.roll(i, 0))
        eager = kb.linear_int8_dynamic(X, W, S)
        g.replay()
        t.cuda.synchronize()
        assert_bits_equal(bits(out), bits(eager), f"replay {i}")

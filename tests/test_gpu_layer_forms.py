"""The kernel forms the layer operators choose between, at sizes where
the choice turned when these were written: the tiles of the int8 product, tokens quantized on the way,
rows by waves or workgroups, several heads a lane group.  (Which kernel of the
product a shape reaches is held in test_int8_choice, with shapes for every
kernel.)  Bars as in
test_gpu_int8 and test_gpu_heads: bits where every rounding is defined, the
oracle's derived bounds for norms and their gradients."""

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer
from tests.gpu_util import assert_bits_equal, assert_f32_bits_equal_nan_as_nan, bits, case, dev, to_dev, torch
from tests.test_gpu_heads import LAYOUTS, assert_close, table_of
from tests.test_gpu_heads import make as make_heads
from tests.test_gpu_int8 import DT, codes_dev, make, product_case, tdt, upload

pytestmark = pytest.mark.gpu


# On 256 compute units, in this order: few rows in pieces of 16 x 16, 32, 48
# and 64, 32 x 32 and 64 (rows x channels), tiles of 64 and 32 x 128, pieces of 64
# x 64, 80 x 48 and 64, tiles of 32, 64, 128 x 128 and 256 x 256, pieces of 112 and
# 128 x 48; most with the last piece of the depth partial.  In the second list it
# is whole: 16 x 32, 48 and 64, 32 x 32 and 64, 16 x 16, tiles of 64, 128, 256 and
# 128 rows, pieces of 112 x 48, tiles of 32 rows.
FORMS = [(1, 7, 20), (1, 4287, 20), (1, 8197, 20), (1, 12393, 20), (17, 6689, 21), (17, 8529, 20), (106, 2351, 128),
         (38, 9511, 640), (49, 12905, 1609), (50, 8657, 1556), (67, 12875, 1982), (36, 152, 256), (139, 10040, 20),
         (321, 8117, 20), (428, 18432, 20), (89, 9166, 2483), (125, 11500, 3001)]
WHOLE = [(2, 4300, 256), (3, 8200, 384), (5, 12400, 512), (20, 6700, 256), (20, 8600, 384), (40, 160, 1024),
         (150, 10040, 512), (333, 8120, 384), (515, 16400, 512), (700, 9000, 640), (110, 11008, 2560), (118, 11659, 2176)]


@pytest.mark.parametrize("i,M,N,K", [(i, *s) for i, s in enumerate(FORMS + WHOLE)])
def test_product_forms(i, M, N, K):
    t = DT[i % 3]
    case(f"linear int8 forms {t} M={M} N={N} K={K}")
    got, want = product_case(M, N, K, t, bias=i % 2 == 0)
    assert_bits_equal(bits(got), want, f"product {M} {N} {K}")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", [(202, 4157, 2276), (128, 2802, 8002), (600, 2100, 3840), (640, 2050, 3300)])
def test_product_with_the_depth_in_parts(t, M, N, K):
    case(f"linear int8 parts {t} M={M} N={N} K={K}")
    need = kb.lib().linear_int8_workspace_bytes(M, N, K)
    assert need > 0 or torch().cuda.get_device_properties(0).multi_processor_count != 256
    got, want = product_case(M, N, K, t, bias=N % 2 == 0)
    assert_bits_equal(bits(got), want, f"product {M} {N} {K}")
    rng = np.random.default_rng(N)
    a, w = (rng.integers(-128, 128, s).astype(np.int8) for s in ((M, K), (N, K)))
    sa, sw = (rng.uniform(1e-3, 1e-2, n).astype(np.float32) for n in (M, N))
    args = codes_dev(a), to_dev(sa), codes_dev(w), to_dev(sw)
    out = torch().full((M, N + 3), 3.0, dtype=tdt(t), device=dev())
    ws = torch().full((max(need, 1),), 171, dtype=torch().uint8, device=dev())
    kb.linear_int8(*args, dtype=tdt(t), out=out[:, 1:N + 1], workspace=ws)
    assert_bits_equal(bits(out[:, 1:N + 1].contiguous()), layer.round_to(layer.product(a, sa, w, sw), t), "out")
    assert (out[:, 0] == 3.0).all() and (out[:, N + 1:] == 3.0).all()
    if need:
        with pytest.raises(ValueError, match="workspace"):
            kb.linear_int8(*args, dtype=tdt(t), workspace=ws[:-1])
    b, x = make(rng, (M, K), t)
    got = kb.linear_int8_dynamic(upload(b, t), *args[2:])
    assert_bits_equal(bits(got), layer.round_to(layer.product(*layer.quantize_rows(x), w, sw), t), "dynamic")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N", [(70, 300), (300, 9000), (600, 9001)])
def test_product_into_rows_of_odd_distance(t, M, N):
    # outputs whose rows do not start at 16 bytes leave the tiles one by one
    case(f"linear int8 odd output rows {t} M={M} N={N}")
    rng = np.random.default_rng(M + N)
    a, w = (rng.integers(-127, 128, s).astype(np.int8) for s in ((M, 300), (N, 300)))
    sa, sw = (rng.uniform(1e-3, 1e-2, n).astype(np.float32) for n in (M, N))
    out = torch().full((M, N + 3), 3.0, dtype=tdt(t), device=dev())
    kb.linear_int8(codes_dev(a), to_dev(sa), codes_dev(w), to_dev(sw), dtype=tdt(t), out=out[:, 1:N + 1])
    assert_bits_equal(bits(out[:, 1:N + 1].contiguous()), layer.round_to(layer.product(a, sa, w, sw), t), "out")
    assert (out[:, 0] == 3.0).all() and (out[:, N + 1:] == 3.0).all()


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", [(4360, 4352, 256), (8200, 2600, 512), (4400, 4362, 256), (2700, 8200, 768), (4360, 4352, 300)])
def test_workgroups_that_take_several_tiles(t, M, N, K):
    # the second and fourth: more tiles of 256 x 256 than compute units, whose
    # workgroups stay; the others run in 128 x 128
    case(f"linear int8 several tiles {t} M={M} N={N} K={K}")
    got, want = product_case(M, N, K, t, bias=M % 100 != 0)
    assert_bits_equal(bits(got), want, f"product {M} {N} {K}")


@pytest.mark.parametrize("M,N,K,px,pw", [(2050, 2049, 131, 131, 133), (2100, 2500, 400, 401, 400), (300, 300, 128, 129, 129),
                                         (70, 200, 2000, 2001, 2003), (1, 5000, 127, 127, 127), (2200, 2300, 17, 17, 17)])
def test_unaligned_rows_in_both_tiles(M, N, K, px, pw):
    for t in DT:
        case(f"linear int8 unaligned {t} M={M} N={N} K={K} strides {px} {pw}")
        got, want = product_case(M, N, K, t, pitches=(px, pw))
        assert_bits_equal(bits(got), want, f"unaligned {t}")


@pytest.mark.parametrize("M,N,K", [(40000, 64, 48), (32769, 300, 20), (70000, 5, 33)])
def test_more_rows_than_a_launch(M, N, K):
    case(f"linear int8 many rows M={M} N={N} K={K}")
    got, want = product_case(M, N, K, "bf16")
    assert_bits_equal(bits(got), want, "rows")


@pytest.mark.parametrize("M", [1, 2, 40])
def test_more_channels_than_a_launch(M):
    N, K = (1 << 20) + 300, 16
    case(f"linear int8 many channels M={M}")
    got, want = product_case(M, N, K, "bf16")
    assert_bits_equal(bits(got), want, "channels")
    rng = np.random.default_rng(M)
    b, x = make(rng, (M, K), "fp16")
    w = rng.integers(-127, 128, (N, K)).astype(np.int8)
    sw = rng.uniform(1e-3, 1e-2, N).astype(np.float32)
    bias = layer.round_to(rng.standard_normal(N).astype(np.float32), "fp16")
    got = kb.linear_int8_dynamic(upload(b, "fp16"), codes_dev(w), to_dev(sw), bias=upload(bias[None], "fp16")[0])
    want = layer.round_to(layer.product(*layer.quantize_rows(x), w, sw, layer.values(bias, "fp16")), "fp16")
    assert_bits_equal(bits(got), want, "dynamic")


@pytest.mark.parametrize("M,N,px,pw", [(5, 20, 1 << 22, 64), (5, 4, 64, 1 << 22), (300, 260, 1 << 22, 64)])
def test_rows_far_apart(M, N, px, pw):
    # from 2^22 bytes between rows on, offsets inside a tile are 64 bits wide
    case(f"linear int8 rows far apart {px} {pw}")
    got, want = product_case(M, N, 50, "fp32", pitches=(px, pw))
    assert_bits_equal(bits(got), want, "far apart")
    if M <= 8:
        rng = np.random.default_rng(1)
        b, x = make(rng, (M, 50), "fp32")
        w = rng.integers(-127, 128, (N, 50)).astype(np.int8)
        sw = rng.uniform(1e-3, 1e-2, N).astype(np.float32)
        got = kb.linear_int8_dynamic(upload(b, "fp32"), codes_dev(w, pw), to_dev(sw))
        assert_bits_equal(bits(got), layer.product(*layer.quantize_rows(x), w, sw).view(np.uint32), "dynamic")


# tokens quantized inside the product: the limits in tokens (8), depth (16384
# for one) and codes together (28 KB), and the three numbers of channels a
# workgroup, with one beyond each
@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", [(1, 300, 16384), (1, 300, 16385), (8, 200, 2048), (9, 200, 2048), (8, 70, 3500),
                                   (8, 70, 3600), (7, 4096, 129), (2, 4097, 500), (3, 12288, 257), (1, 12289, 640),
                                   (8, 13000, 100), (4, 1, 1), (8, 17, 127)])
def test_tokens(t, M, N, K):
    case(f"linear int8 tokens {t} M={M} N={N} K={K}")
    rng = np.random.default_rng(M * N + K)
    whole, _ = make(rng, (M, K + 1), t)
    w = rng.integers(-128, 128, (N, K)).astype(np.int8)
    sw = rng.uniform(1e-3, 1e-2, N).astype(np.float32)
    W, S = codes_dev(w), to_dev(sw)
    for lo in (0, 1):  # rows of K + 1 elements: aligned and not
        b = whole[:, lo:lo + K]
        X = upload(whole, t)[:, lo:lo + K]
        want = layer.round_to(layer.product(*layer.quantize_rows(layer.values(b, t)), w, sw), t)
        assert_bits_equal(bits(kb.linear_int8_dynamic(X, W, S)), want, f"from column {lo}")
        assert_bits_equal(bits(kb.linear_int8_dynamic(X.contiguous(), W, S)), want, "contiguous")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("rows,d", [(1021, 200), (1025, 4096), (1024, 4097), (1030, 513), (1022, 4091), (3000, 8), (5000, 1)])
def test_many_rows_to_codes(t, rows, d):
    case(f"int8 rows {t} {rows}x{d}")
    b, _ = make(np.random.default_rng(rows + d), (rows, d + 3), t)
    b[5] = 0
    b[6, d // 2 + 1] = {"fp32": 0x7FC00000, "fp16": 0x7E00, "bf16": 0x7FC0}[t]
    b[rows - 1, d] = {"fp32": 0xFF800000, "fp16": 0xFC00, "bf16": 0xFF80}[t]
    for lo in (0, 1):
        part = b[:, lo:lo + d]
        X = upload(b, t)[:, lo:lo + d]
        q, s = layer.quantize_rows(layer.values(part, t))
        for x in (X, X.contiguous()):
            codes, scale = kb.quantize_rows_int8(x)
            assert np.array_equal(codes.cpu().numpy(), q)
            assert_f32_bits_equal_nan_as_nan(bits(scale), s.view(np.uint32), "scale")
            pitch = -(-d // 16) * 16
            assert not torch().as_strided(codes, (rows, pitch), (pitch, 1)).cpu().numpy()[:, d:].any()


# several heads a lane group, with heads left over, in each way a row is held:
# pieces of 8, one pair a lane, 8 pairs a lane
LARGE = [(3001, 7, 128, 128), (2501, 5, 64, 32), (3000, 3, 72, 40), (2000, 5, 100, 50), (700, 3, 200, 66), (6000, 1, 256, 256)]


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H,D,rot", LARGE)
def test_rope_large(t, layout, T, H, D, rot):
    case(f"rope {t} {layout} T={T} H={H} D={D} rot={rot}")
    rng = np.random.default_rng(T + H + D)
    b, x = make_heads(rng, (T, H, D), t)
    table, tab = table_of(rot, 777)
    pos = rng.integers(0, 777, T)
    want = layer.round_to(layer.rotate(x, pos, tab, layout), t)
    v = upload(b, t)
    assert_bits_equal(bits(kb.rope(v, to_dev(pos), table, layout=layout)), want, "tokens' heads together")
    head_major = v.transpose(0, 1).contiguous().transpose(0, 1)
    kb.rope(head_major, to_dev(pos), table, layout=layout, out=head_major)
    assert_bits_equal(bits(head_major.contiguous()), want, "heads' tokens together, in place")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H,D,rot", LARGE)
def test_norm_and_gradient_large(t, layout, T, H, D, rot):
    case(f"norm {t} {layout} T={T} H={H} D={D} rot={rot}")
    rng = np.random.default_rng(T + H + D + 1)
    Hk = (H + 1) // 2
    table, tab = table_of(rot, 777)
    pos = rng.integers(0, 777, T)
    eps = float(np.float32(1e-6))
    one = {}
    for n, h in (("q", H), ("k", Hk)):
        one[n] = make_heads(rng, (T, h, D), t, 2.0), make_heads(rng, (T, h, D), t), make_heads(rng, (D,), t)
    up = {n: [upload(v[0][0], t), upload(v[1][0], t), upload(v[2][0][None], t)[0]] for n, v in one.items()}
    out = kb.qk_norm_rope(up["q"][0], up["k"][0], up["q"][2], up["k"][2], to_dev(pos), table, layout=layout)
    back = kb.qk_norm_rope_backward(up["q"][1], up["k"][1], up["q"][0], up["k"][0], up["q"][2], up["k"][2],
                                    to_dev(pos), table, layout=layout)
    for i, n in enumerate("qk"):
        (_, x), (_, g), (_, w) = one[n]
        assert_close(bits(out[i]), t, *layer.norm_rope(x, w, pos, tab, eps, layout), n)
        dx, dxb, dw, dwb = layer.norm_rope_back(g, x, w, pos, tab, eps, layout)
        assert_close(bits(back[i]), t, dx, dxb, "d" + n)
        assert_close(bits(back[2 + i]), "fp32", dw, dwb, f"d{n}_weight")


@pytest.mark.parametrize("rows", [15, 16, 17, 31, 32, 33, 63, 64, 65, 66, 127, 128, 129, 200])
def test_norm_gradient_with_and_without_the_second_kernel(rows):
    # heads of 128 in 16 bits: 8 lanes a row, 32 rows a workgroup, or 128 in one
    # large workgroup a set, which stores its sums directly
    for H, Hk in ((4, 1), (2, 2), (1, 3)):
        case(f"norm gradient rows={rows} heads={H},{Hk}")
        rng = np.random.default_rng(rows + H)
        table, tab = table_of(128, 64)
        pos = rng.integers(0, 64, rows)
        eps = float(np.float32(1e-6))
        (xb, x), (gb, g), (wb, w) = (make_heads(rng, s, "bf16") for s in ((rows, H, 128), (rows, H, 128), (128,)))
        (yb, y), (hb, h) = (make_heads(rng, (rows, Hk, 128), "bf16") for _ in range(2))
        W = upload(wb[None], "bf16")[0]
        got = kb.qk_norm_rope_backward(upload(gb, "bf16"), upload(hb, "bf16"), upload(xb, "bf16"), upload(yb, "bf16"),
                                       W, W, to_dev(pos), table)
        for i, (a, b) in enumerate(((g, x), (h, y))):
            dx, dxb, dw, dwb = layer.norm_rope_back(a, b, w, pos, tab, eps, "half")
            assert_close(bits(got[i]), "bf16", dx, dxb, "dx")
            assert_close(bits(got[2 + i]), "fp32", dw, dwb, "dw")


def test_gradients_of_broadcast_heads():
    # one gradient for all heads (stride 0), as the backward of a sum over them gives
    t = torch()
    rng = np.random.default_rng(4)
    T, H, D = 40, 6, 64
    (xb, x), (gb, g), (wb, w) = (make_heads(rng, s, "bf16") for s in ((T, H, D), (T, 1, D), (D,)))
    table, tab = table_of(64, 64)
    pos = np.arange(T)
    W, X, G = upload(wb[None], "bf16")[0], upload(xb, "bf16"), upload(gb, "bf16").expand(T, H, D)
    case("norm gradient, broadcast")
    dq, dk, dqw, dkw = kb.qk_norm_rope_backward(G, G[:, :2], X, X[:, :2], W, W, to_dev(pos), table)
    dx, dxb, dw, dwb = layer.norm_rope_back(np.broadcast_to(g, x.shape), x, w, pos, tab, float(np.float32(1e-6)), "half")
    assert_close(bits(dq), "bf16", dx, dxb, "dq")
    assert_close(bits(dqw), "fp32", dw, dwb, "dq_weight")
    case("rope gradient, broadcast")
    got = kb.rope(G, to_dev(pos), table, inverse=True)
    want = layer.round_to(layer.rotate(np.broadcast_to(g, x.shape), pos, tab, "half", True), "bf16")
    assert_bits_equal(bits(got), want, "rope")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("T,H,D,Dv,rot,page", [(4001, 5, 128, 128, 128, 16), (3500, 6, 64, 128, 32, 7), (3000, 3, 72, 50, 40, 32)])
def test_append_large(t, T, H, D, Dv, rot, page):
    case(f"append {t} T={T} H={H} D={D} Dv={Dv} rot={rot} page={page}")
    rng = np.random.default_rng(T + H)
    pages = -(-T // page) + 3
    (kb_, k), (vb, _) = make_heads(rng, (T, H, D), t), make_heads(rng, (T, H, Dv), t)
    kcb, _ = make_heads(rng, (pages, page, H, D), t)
    vcb, _ = make_heads(rng, (pages, page, H, Dv), t)
    slots = rng.permutation(pages * page)[:T]
    slots[::17] = -1
    pos = rng.integers(0, 300, T)
    table, tab = table_of(rot, 300)
    caches = [upload(c, t) for c in (kcb, vcb)]
    kb.append_kv_paged(upload(kb_, t), upload(vb, t), to_dev(slots), *caches, positions=to_dev(pos), table=table)
    rows = layer.round_to(layer.rotate(k, pos, tab, "half"), t)
    assert_bits_equal(bits(caches[0]), layer.append(kcb, rows, slots), "k_cache")
    assert_bits_equal(bits(caches[1]), layer.append(vcb, vb, slots), "v_cache")

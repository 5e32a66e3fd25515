"""GPU parity of the int8 product in every kernel the rule picks from, at
depths that run its loops to the end; tests/test_int8_choice.py holds which
kernel each shape reaches.  The bar is bit equality with the oracle."""

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer
from tests.gpu_util import assert_bits_equal, bits, case, dev, to_dev, torch
from tests.test_gpu_int8 import DT, codes_dev, product_case, tdt
from tests.test_int8_choice import FEW, LARGE, PARTS, STAY, TILES

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("i,M,N,K", [(i, *s[1:]) for i, s in enumerate(FEW + TILES)])
def test_few_rows_and_tiles(i, M, N, K):
    for t in (DT[i % 3], DT[(i + 1) % 3]):
        case(f"linear int8 {t} M={M} N={N} K={K}")
        got, want = product_case(M, N, K, t, bias=t == DT[i % 3])
        assert_bits_equal(bits(got), want, f"product {t} {M} {N} {K}")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", LARGE + STAY)
def test_large_tiles(t, M, N, K):
    case(f"linear int8 large tiles {t} M={M} N={N} K={K}")
    got, want = product_case(M, N, K, t, bias=M % 3 != 0)
    assert_bits_equal(bits(got), want, f"product {M} {N} {K}")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("parts,M,N,K", PARTS)
def test_parts(t, parts, M, N, K):
    case(f"linear int8 {parts} parts {t} M={M} N={N} K={K}")
    got, want = product_case(M, N, K, t, bias=N % 2 != 0)
    assert_bits_equal(bits(got), want, f"product {M} {N} {K}")


@pytest.mark.parametrize("t", DT)
def test_large_tiles_into_rows_of_odd_distance(t):
    # a shape whose workgroups would stay: not with rows of outputs that start anywhere
    M, N, K = STAY[2]
    case(f"linear int8 large tiles, odd output rows {t}")
    rng = np.random.default_rng(M)
    a, w = (rng.integers(-128, 128, s).astype(np.int8) for s in ((M, K), (N, K)))
    sa, sw = (rng.uniform(1e-3, 1e-2, n).astype(np.float32) for n in (M, N))
    out = torch().full((M, N + 3), 3.0, dtype=tdt(t), device=dev())
    kb.linear_int8(codes_dev(a), to_dev(sa), codes_dev(w), to_dev(sw), dtype=tdt(t), out=out[:, 1:N + 1])
    assert_bits_equal(bits(out[:, 1:N + 1].contiguous()), layer.round_to(layer.product(a, sa, w, sw), t), "out")
    assert (out[:, 0] == 3.0).all() and (out[:, N + 1:] == 3.0).all()


def test_one_workspace_for_every_batch():
    # 171 x 5815 x 4096 puts its depth in parts, the others do not
    N, K = PARTS[2][2:]
    t = torch()
    ws = t.empty(kb.lib().linear_int8_workspace_bytes(2048, N, K), dtype=t.uint8, device=dev())
    wd = t.empty(kb.lib().linear_int8_dynamic_workspace_bytes(2048, N, K), dtype=t.uint8, device=dev())
    rng = np.random.default_rng(3)
    w = rng.integers(-127, 128, (N, K)).astype(np.int8)
    sw = rng.uniform(1e-3, 1e-2, N).astype(np.float32)
    x = rng.standard_normal((600, K)).astype(np.float32)
    W, S, X = codes_dev(w), to_dev(sw), to_dev(x)
    q, s = layer.quantize_rows(x)
    Q, SX = codes_dev(q), to_dev(s)
    want = layer.product(q, s, w, sw).view(np.uint32)
    for M in (600, 171, 256, 64, 1):
        case(f"linear int8 one workspace M={M}")
        assert_bits_equal(bits(kb.linear_int8(Q[:M], SX[:M], W, S, dtype=t.float32, workspace=ws)), want[:M], "codes")
        assert_bits_equal(bits(kb.linear_int8_dynamic(X[:M], W, S, workspace=wd)), want[:M], "values")

"""GPU parity of int8 products with one row of codes on either side, whose
depth is no multiple of 16: aligned operands, although no distance of rows
says so.  The bar is bit equality with the oracle."""

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer
from tests.gpu_util import assert_bits_equal, bits, case, to_dev
from tests.test_gpu_int8 import DT, codes_dev, make, product_case, upload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,N,K", [(1, 4096, 3000), (1, 300, 4095), (1, 12300, 1001), (1, 64, 2), (1, 1, 1), (1, 1, 5003),
                                   (2, 1, 130), (70, 1, 4095), (3000, 1, 999), (33000, 1, 17)])
def test_product(t, M, N, K):
    case(f"linear int8 single row {t} M={M} N={N} K={K}")
    got, want = product_case(M, N, K, t, bias=N > 1)
    assert_bits_equal(bits(got), want, f"product {M} {N} {K}")


@pytest.mark.parametrize("t", DT)
@pytest.mark.parametrize("M,K", [(1, 3000), (1, 17), (8, 3333), (5, 129), (12, 4001)])
def test_tokens_on_a_single_channel(t, M, K):
    case(f"linear int8 dynamic single channel {t} M={M} K={K}")
    rng = np.random.default_rng(M + K)
    b, x = make(rng, (M, K), t)
    w = rng.integers(-128, 128, (1, K)).astype(np.int8)
    sw = rng.uniform(1e-3, 1e-2, 1).astype(np.float32)
    want = layer.round_to(layer.product(*layer.quantize_rows(x), w, sw), t)
    for pitch in (None, K, 1 << 22):
        got = kb.linear_int8_dynamic(upload(b, t), codes_dev(w, pitch), to_dev(sw))
        assert_bits_equal(bits(got), want, f"distance {pitch}")

"""Arguments the layer operators' binding refuses, and their close neighbours
that it takes."""

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer
from tests.gpu_util import assert_bits_equal, bits, case, dev, to_dev, torch
from tests.test_gpu_int8 import codes_dev

pytestmark = pytest.mark.gpu


def test_vectors_of_another_layer():
    t = torch()
    rng = np.random.default_rng(1)
    a, w = rng.integers(-127, 128, (3, 32)).astype(np.int8), rng.integers(-127, 128, (5, 32)).astype(np.int8)
    sa, sw = rng.uniform(0.1, 1, 4).astype(np.float32), rng.uniform(0.1, 1, 6).astype(np.float32)
    bias = t.ones(6, device=dev())
    A, W, SA, SW = codes_dev(a), codes_dev(w), to_dev(sa), to_dev(sw)
    x = t.ones(3, 32, device=dev())
    for fn in (lambda s, b: kb.linear_int8(A, SA, W, s, bias=b, dtype=t.float32),
               lambda s, b: kb.linear_int8_dynamic(x, W, s, bias=b)):
        case("int8 vectors of another layer")
        with pytest.raises(ValueError, match="w_scale: 6 elements for 5 channels"):
            fn(SW, None)
        with pytest.raises(ValueError, match="w_scale: 4 elements"):
            fn(SW[:4], None)
        with pytest.raises(ValueError, match="bias: 6 elements for 5 channels"):
            fn(SW[:5], bias)
        fn(SW[:5], bias[:5])
        fn(SW[:5, None], bias[None, :5])  # one value a channel, in any shape
    # a vector of rows' scales may be longer, as the one that quantize_rows_int8 may be given
    got = kb.linear_int8(A, SA, W, SW[:5], dtype=t.float32)
    assert_bits_equal(bits(got), layer.product(a, sa[:3], w, sw[:5]).view(np.uint32), "longer scale")

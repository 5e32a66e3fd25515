"""Bit equality of MXFP4 products on shapes that reach every kernel form's loops
(tests/test_mx_choice.py holds the rule to them)."""

import numpy as np
import pytest

import blockwise_bit_codebook_amd as kb
from oracle import layer, mx
from tests.gpu_util import assert_bits_equal, bits, case, torch
from tests.test_gpu_int8 import DT, tdt, upload
from tests.test_gpu_mxfp4 import random_codes, u8
from tests.test_mx_choice import FEW, LARGE, PARTS, RING

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,M,N,K", [(f"few {p}", *s) for p, *s in FEW] + [(f"ring {b} {st}", *s) for b, st, *s in RING] +
                         [("256", *s) for s in LARGE] + [(f"parts {p} {st}", *s) for p, st, *s in PARTS])
def test_forms(form, M, N, K):
    # with all scales 1 sums are multiples of 1/4 below 36 K < 2^20, and a bias of
    # quarters: fp32 holds every partial sum in any order
    t = DT[(M + N + K) % 3]
    rng = np.random.default_rng(M + 5 * N + 7 * K)
    a, w = random_codes(rng, M, K, 127, 127), random_codes(rng, N, K, 127, 127)
    # some rows and channels at other powers of two: those sums scale as a whole
    a[1][::3], w[1][::5] = 125, 130
    y = mx.values(*a).astype(np.float32) @ mx.values(*w).astype(np.float32).T
    bb = None
    if (M + N) % 2:
        bb = layer.round_to((rng.integers(-64, 65, N) / 4).astype(np.float32), t)
        y = y + layer.values(bb, t).astype(np.float32)
    case(f"linear mxfp4 {form} {t} M={M} N={N} K={K}")
    got = kb.linear_mxfp4(u8(a[0]), u8(a[1]), u8(w[0]), u8(w[1]), bias=None if bb is None else upload(bb[None], t)[0],
                          dtype=tdt(t))
    assert_bits_equal(bits(got), layer.round_to(y, t), f"{form} {M} {N} {K}")
    torch().cuda.empty_cache()

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


def brute(x, y=None):
    """Whether two rows (last axis) share an element: of x and y, or two of x."""
    def rows(v):
        t = torch().as_strided(torch().arange(v.untyped_storage().nbytes() // v.element_size()), v.shape, v.stride(),
                               v.storage_offset())
        return t.reshape(-1, v.shape[-1]).numpy()
    a = rows(x)
    if y is None:
        return np.unique(a).size < a.size
    return bool(np.intersect1d(a, rows(y)).size)


def test_outputs_that_overlap():
    # views of one buffer with random sizes, strides and starts: an output is
    # refused exactly where two of its rows, or one of its and one of the
    # input's (unless it is the input), share elements
    t = torch()
    freq, _ = kb.rope_frequencies(4)
    table = kb.rope_table(freq, 8)
    rng = np.random.default_rng(2)
    buf = t.zeros(400, device=dev())
    refused = taken = 0
    for i in range(600):
        B, T, H = (int(v) for v in rng.integers(1, 5, 3))
        D = 4

        def view(like=None):
            while True:
                nested = sorted(int(v) for v in rng.integers(1, 30, 3)) if rng.random() < 0.5 else \
                    [D + int(rng.integers(0, 2)), (D + 1) * H, (D + 1) * H * T + int(rng.integers(0, 8))]
                st = like.stride()[:3] if like is not None and rng.random() < 0.6 else \
                    tuple(int(v) for v in (rng.permutation(nested) if rng.random() < 0.3 else nested[::-1]))
                at = int(rng.integers(0, 60)) if like is None or rng.random() < 0.8 else like.storage_offset()
                if at + sum((n - 1) * s for n, s in zip((B, T, H), st)) + D <= buf.numel():
                    return t.as_strided(buf, (B, T, H, D), (*st, 1), at)
        x = view()
        out = view(x)
        pos = t.zeros((B, T), dtype=t.int64, device=dev())
        same = x.data_ptr() == out.data_ptr() and x.stride() == out.stride()
        want = brute(out) or (brute(x, out) and not same)
        if want:
            refused += 1
            with pytest.raises(ValueError, match="overlap"):
                kb.rope(x, pos, table, out=out)
        else:
            taken += 1
            kb.rope(x, pos, table, out=out)
    assert refused > 100 and taken > 100, (refused, taken)


def test_outputs_over_the_other_operand():
    t = torch()
    freq, _ = kb.rope_frequencies(64)
    table, w = kb.rope_table(freq, 8), t.ones(64, device=dev())
    pos = t.zeros(6, dtype=t.int64, device=dev())
    qkv = t.ones(6, 8 * 64, device=dev())
    q, k, v = (qkv[:, a * 64:b * 64].view(6, b - a, 64) for a, b in ((0, 4), (4, 6), (6, 8)))
    over = qkv[:, 3 * 64:7 * 64].view(6, 4, 64)  # one head of q, those of k and one of v

    def forward(**kw):
        return kb.qk_norm_rope(q, k, w, w, pos, table, **kw)

    def back(gq, gk, **kw):
        return kb.qk_norm_rope_backward(gq, gk, q, k, w, w, pos, table, **kw)

    for fn, match in ((lambda: forward(q_out=over), "q_out overlaps q"),
                      (lambda: forward(k_out=over[:, :2]), "k_out overlaps k"),
                      (lambda: forward(k_out=q[:, 1:3]), "k_out overlaps q"),
                      (lambda: forward(q_out=q[:, :1].expand(6, 4, 64)), "q_out: elements overlap"),
                      (lambda: forward(q_out=t.as_strided(qkv, (6, 4, 64), (512, 32, 1))), "q_out: elements overlap"),
                      (lambda: back(t.ones_like(q), k.clone(), dq=over), "dq overlaps q"),
                      (lambda: back(over, k.clone(), dq=qkv[:, 2 * 64:6 * 64].view(6, 4, 64)), "dq overlaps"),
                      (lambda: back(t.ones_like(q), over[:, 2:], dk=v), "dk overlaps dk_out"),
                      (lambda: kb.linear_int8_dynamic(qkv[:, :64], codes_dev(np.ones((64, 64), np.int8)), w,
                                                      out=qkv[:, 32:96]), "out overlaps X")):
        case(f"overlap: {match}")
        with pytest.raises(ValueError, match=match):
            fn()
    new = t.empty(6, 6, 64, device=dev())
    with pytest.raises(ValueError, match="q_out overlaps k_out"):
        forward(q_out=new[:, :4], k_out=new[:, 3:5])
    # neighbours in one buffer do not overlap
    forward(q_out=q, k_out=v)
    forward(q_out=new[:, :4], k_out=new[:, 4:])
    forward(q_out=q, k_out=k)
    g = t.ones(6, 6, 64, device=dev())
    back(g[:, :4], g[:, 4:], dq=g[:, :4], dk=g[:, 4:])
    kb.linear_int8_dynamic(qkv[:, :64], codes_dev(np.ones((64, 64), np.int8)), w, out=qkv[:, 64:128])
    kb.rope(q, pos, table, out=qkv[:, 4 * 64:].view(6, 4, 64))

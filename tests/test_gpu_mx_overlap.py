"""Operands and outputs of the MXFP4 operators and of the layer norm in one
buffer: rows that lie between each other's are used as they are, rows that
share a byte are refused."""

import pytest

import blockwise_bit_codebook_amd as kb
from tests.gpu_util import assert_bits_equal, bits, case, dev, torch

pytestmark = pytest.mark.gpu

M, N, K = 8, 16, 64  # two blocks a row: 32 bytes of codes, 2 of scales


class Buffer:
    """Rows of `pitch` bytes; view(): matrices of a type in them, at a byte of a row."""

    def __init__(self, rows, pitch):
        self.pitch = pitch
        self.bytes = torch().full((rows * pitch + 64,), 0xEE, dtype=torch().uint8, device=dev())

    def view(self, dtype, rows, cols, at, pitch=None):
        flat = self.bytes.view(dtype)
        size = flat.element_size()
        assert at % size == 0 and self.pitch % size == 0
        return torch().as_strided(flat, (rows, cols), ((pitch or self.pitch) // size, 1), at // size)


def filled(view, seed=0):
    g = torch().Generator().manual_seed(seed)
    view.copy_(torch().randn(view.shape, generator=g).to(dev()))
    return view


def same(got, want, what):
    for g, w in zip(got, want):
        assert_bits_equal(bits(g.contiguous()), bits(w.contiguous()), what)


def bad(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


@pytest.mark.parametrize("name", ["float32", "float16", "bfloat16"])
def test_codes_beside_the_values(name):
    T = torch()
    t = getattr(T, name)
    size = K * T.empty(0, dtype=t).element_size()
    b = Buffer(M, size + 48)
    x = filled(b.view(t, M, K, 0))
    case(f"mx overlap: codes beside {name} values")
    want = kb.quantize_mxfp4(x.clone())
    given = b.view(T.uint8, M, 32, size), b.view(T.uint8, M, 2, size + 32)
    same(kb.quantize_mxfp4(x, *given), want, "rows")
    back = kb.dequantize_mxfp4(*want, K, dtype=t)
    out = b.view(t, M, K, 0)  # the values' own place
    kb.dequantize_mxfp4(*given, K, dtype=t, out=out)
    same([out], [back], "values")
    # one byte too far
    bad("codes overlaps X", kb.quantize_mxfp4, x, b.view(T.uint8, M, 32, size - 1), given[1])
    bad("scales overlaps X", kb.quantize_mxfp4, x, given[0], b.view(T.uint8, M, 2, size + 47))  # the last into the next row
    bad("out overlaps scales", kb.dequantize_mxfp4, given[0], b.view(T.uint8, M, 2, size - 1), K, dtype=t, out=out)
    bad("out overlaps codes", kb.dequantize_mxfp4, b.view(T.uint8, M, 32, size - 16), given[1], K, dtype=t, out=out)
    # rows twice as far apart, in the first half of the buffer's
    few = b.view(T.uint8, M // 2, 32, size, 2 * b.pitch), b.view(T.uint8, M // 2, 2, size + 32, 2 * b.pitch)
    same(kb.quantize_mxfp4(x[M // 2:], *few), [w[M // 2:] for w in want], "every other row")
    bad("codes overlaps X", kb.quantize_mxfp4, x[M // 2:], b.view(T.uint8, M // 2, 32, size - 16, 2 * b.pitch), few[1])


def test_codes_beside_the_columns():
    # X.t(): 8 columns of 64 values, their codes in the gaps of X's first rows
    T = torch()
    b = Buffer(K, 2 * M + 48)
    x = filled(b.view(T.bfloat16, K, M, 0))
    given = b.view(T.uint8, M, 32, 2 * M), b.view(T.uint8, M, 2, 2 * M + 32)
    case("mx overlap: codes beside columns")
    want = kb.quantize_mxfp4(x.t().contiguous())
    same(kb.quantize_mxfp4(x.t(), *given), want, "columns")
    bad("codes overlaps X", kb.quantize_mxfp4, x.t(), b.view(T.uint8, M, 32, 2 * M - 1), given[1])
    bad("scales overlaps X", kb.quantize_mxfp4, x.t(), given[0], b.view(T.uint8, M, 2, 2 * M + 47))
    bad("codes overlaps X", kb.quantize_mxfp4, x.t(), b.bytes[-M * 32:].view(M, 32), given[1])


def test_products_into_the_operands_buffer():
    T = torch()
    f32 = T.float32
    x, w = filled(T.empty(M, K, device=dev())), filled(T.empty(N, K, device=dev()), 1)
    bias = filled(T.empty(1, N, device=dev()), 2)[0]
    b = Buffer(N, 48 + 4 * N)
    wc, ws = kb.quantize_mxfp4(w, b.view(T.uint8, N, 32, 0), b.view(T.uint8, N, 2, 32))
    xc, xs = kb.quantize_mxfp4(x)
    want = kb.linear_mxfp4(xc, xs, wc.contiguous(), ws.contiguous(), bias=bias, dtype=f32)
    # the bias behind the last row of outputs
    held = b.view(f32, N, N, 48)
    held[M].copy_(bias)
    case("mx overlap: products into the weight's buffer")
    kb.linear_mxfp4(xc, xs, wc, ws, bias=held[M], dtype=f32, out=held[:M])
    same([held[:M]], [want], "codes")
    kb.linear_mxfp4_dynamic(x, wc, ws, bias=held[M], out=held[:M])
    same([held[:M]], [want], "values")
    for fn in (lambda out, bias=None: kb.linear_mxfp4(xc, xs, wc, ws, bias=bias, dtype=f32, out=out),
               lambda out, bias=None: kb.linear_mxfp4_dynamic(x, wc, ws, bias=bias, out=out)):
        bad("out overlaps w_codes", fn, b.view(f32, M, N, 28))
        bad("out overlaps w_scales", fn, b.view(f32, M, N, 32))
        bad("out overlaps w_codes", fn, b.view(f32, M, N, 52))      # the last channel into the next row
        bad("out overlaps bias", fn, held[:M], held[M - 1])
    bad("out overlaps scales", kb.linear_mxfp4, xc, b.bytes[48:48 + 2 * M].view(M, 2), wc, ws, dtype=f32, out=held[:M])


def test_gradients_beside_the_operands():
    T = torch()
    g, x, w = (filled(T.empty(s, device=dev()), i) for i, s in enumerate(((M, N), (M, K), (N, K))))
    want = kb.linear_mxfp4_backward(g, x, w)
    b = Buffer(N, 4 * (3 * K + N))
    at = [0, 4 * K, 8 * K, 12 * K]
    bg, bx, bw = b.view(T.float32, M, N, at[3]), b.view(T.float32, M, K, at[1]), b.view(T.float32, N, K, at[0])
    bg.copy_(g), bx.copy_(x), bw.copy_(w)
    dw, dx = b.view(T.float32, N, K, at[2]), b.view(T.float32, N, K, at[1])[M:]  # dX in the rows that X leaves
    case("mx overlap: gradients beside the operands")
    got = kb.linear_mxfp4_backward(bg, bx, bw, dX=dx, dweight=dw)
    same(got, want, "gradients")
    bad("dweight overlaps dout", kb.linear_mxfp4_backward, bg, bx, bw, dweight=b.view(T.float32, N, K, at[2] + 4))
    bad("dweight overlaps X", kb.linear_mxfp4_backward, bg, bx, bw, dweight=b.view(T.float32, N, K, at[2] - 4))
    bad("dweight overlaps weight", kb.linear_mxfp4_backward, bg, x, bw, dweight=b.view(T.float32, N, K, 4))
    bad("dweight overlaps dX", kb.linear_mxfp4_backward, g, x, w, dX=dx, dweight=b.view(T.float32, N, K, at[2] - 4))


def test_norm_beside_its_weights():
    T = torch()
    x = filled(T.empty(M, K, device=dev(), dtype=T.bfloat16))
    w, nb = filled(T.empty(1, K, device=dev()), 1)[0], filled(T.empty(1, K, device=dev()), 2)[0]
    want = kb.layer_norm(x, w, nb)
    dwant = kb.layer_norm_backward(x, x.clone(), w)
    b = Buffer(M, 2 * K + 4 * K)
    out = b.view(T.bfloat16, M, K, 0)
    hw, hb = b.view(T.float32, M, K, 2 * K)[2], b.view(T.float32, M, K, 2 * K)[M - 2]
    hw.copy_(w), hb.copy_(nb)
    case("mx overlap: norm beside its weights")
    same([kb.layer_norm(x, hw, hb, out=out)], [want], "norm")
    same(kb.layer_norm_backward(x, x.clone(), hw, dx=out), dwant, "gradient")
    off = b.bytes.view(T.float32)[2 * b.pitch // 4 + K // 2 - 1:][:K]  # from the last values of a row on
    bad("out overlaps weight", kb.layer_norm, x, off, hb, out=out)
    bad("out overlaps bias", kb.layer_norm, x, hw, off, out=out)
    bad("dx overlaps weight", kb.layer_norm_backward, x, x.clone(), off, dx=out)
    # weights of another shape than one row
    same([kb.layer_norm(x, hw.view(2, 2, 2, 2, 2, 2), hb.view(K, 1), out=out)], [want], "shapes")


def test_thousands_of_rows_at_two_distances():
    T = torch()
    b = Buffer(6000, 256)
    x = filled(b.view(T.bfloat16, 6000, K, 0))
    want = kb.quantize_mxfp4(x[:3000].clone())
    scales = T.empty(3000, 2, dtype=T.uint8, device=dev())
    case("mx overlap: rows at two distances")
    codes = b.view(T.uint8, 3000, 32, 128, 512)  # beside every other row of x
    same(kb.quantize_mxfp4(x[:3000], codes, scales), want, "beside")
    codes = b.view(T.uint8, 3000, 32, 128, 496)  # 16 bytes nearer from row to row: the second one meets the third of x
    bad("codes overlaps X", kb.quantize_mxfp4, x[:3000], codes, scales)
    same([scales], want[1:], "left alone")


def test_workspaces_that_hold_a_tensor_of_the_call():
    T, lib = torch(), kb.lib()
    rows, n, k = 300, 256, 2048
    t = T.bfloat16
    x, g, w = (filled(T.empty(s, device=dev(), dtype=t), i) for i, s in enumerate(((rows, k), (rows, n), (n, k))))
    wq, xq = kb.quantize_mxfp4(w), kb.quantize_mxfp4(x)
    bias, out = T.zeros(n, device=dev(), dtype=t), T.empty(rows, n, device=dev(), dtype=t)
    space = T.full((16 << 20,), 0xFF, dtype=T.uint8, device=dev())

    def inside(v, at):  # a copy of v in the workspace's bytes
        held = space[at:at + v.numel() * v.element_size()].view(v.dtype).view(v.shape)
        return held.copy_(v)
    case("mx overlap: workspaces")
    # the values' codes are the first thing there
    need = lib.linear_mxfp4_dynamic_workspace_bytes(rows, n, k)
    want = kb.linear_mxfp4_dynamic(x, *wq, bias=bias)
    for name, kw in (("X", dict(x=inside(x, 0))), ("w_codes", dict(c=inside(wq[0], 16))), ("w_scales", dict(s=inside(wq[1], 3))),
                     ("bias", dict(bias=inside(bias, 2))), ("out", dict(out=inside(out, 64)))):
        a = dict(dict(x=x, c=wq[0], s=wq[1], bias=bias, out=out), **kw)
        bad(f"workspace overlaps {name}", kb.linear_mxfp4_dynamic, a["x"], a["c"], a["s"], bias=a["bias"], out=a["out"], workspace=space)
    same([kb.linear_mxfp4_dynamic(inside(x, need), inside(wq[0], 8 << 20), wq[1], bias=bias, workspace=space)], [want], "behind its use")
    few = kb.linear_mxfp4_dynamic(inside(x[:4], 0), *wq, workspace=space)  # nothing of it is used
    same([few], [kb.linear_mxfp4_dynamic(x[:4], *wq)], "tokens")
    # gradients
    need = lib.linear_mxfp4_backward_workspace_bytes(rows, n, k)
    want = kb.linear_mxfp4_backward(g, x, w)
    for name, kw in (("dout", dict(g=inside(g, 0))), ("X", dict(x=inside(x, 2))), ("weight", dict(w=inside(w, 16)))):
        a = dict(dict(g=g, x=x, w=w), **kw)
        bad(f"workspace overlaps {name}", kb.linear_mxfp4_backward, a["g"], a["x"], a["w"], workspace=space)
    bad("workspace overlaps dX", kb.linear_mxfp4_backward, g, x, w, dX=inside(x, 0), workspace=space)
    bad("workspace overlaps dweight", kb.linear_mxfp4_backward, g, x, w, dweight=inside(w.float(), 0), workspace=space)
    assert need + x.numel() * 2 + w.numel() * 4 < space.numel()
    got = kb.linear_mxfp4_backward(g, inside(x, need), w, dweight=inside(w.float(), need + x.numel() * 2), workspace=space)
    same(got, want, "behind its use")
    # norm
    nw = T.ones(k, device=dev())
    for name, kw in (("dout", dict(g=inside(x, 0))), ("x", dict(x=inside(x, 0))), ("weight", dict(w=inside(nw, 4)))):
        a = dict(dict(g=x.clone(), x=x, w=nw), **kw)
        bad(f"workspace overlaps {name}", kb.layer_norm_backward, a["g"], a["x"], a["w"], workspace=space)
    bad("workspace overlaps dx", kb.layer_norm_backward, x.clone(), x, nw, dx=inside(x, 0), workspace=space)
    # sums of parts of the depth
    a, w = T.zeros(1005, 8112, dtype=T.uint8, device=dev()), T.zeros(1301, 8112, dtype=T.uint8, device=dev())
    sa, sw = T.zeros(1005, 507, dtype=T.uint8, device=dev()), T.zeros(1301, 507, dtype=T.uint8, device=dev())
    space = T.empty(lib.linear_mxfp4_workspace_bytes(1005, 1301, 16224), dtype=T.uint8, device=dev())
    for name, args in (("codes", (inside(a, 0), sa, w, sw)), ("scales", (a, inside(sa, 0), w, sw)), ("w_codes", (a, sa, inside(w, 0), sw)),
                       ("w_scales", (a, sa, w, inside(sw, 0)))):
        bad(f"workspace overlaps {name}", kb.linear_mxfp4, *args, workspace=space)

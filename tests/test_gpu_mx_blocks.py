"""Bit equality of MXFP4 products and gradients of more rows or channels than one
launch takes (tests/test_mx_blocks.py holds which kernel each block reaches), in
workspaces that are full of NaN scales and end where the library says."""

import pytest

import blockwise_bit_codebook_amd as kb
from tests.gpu_util import case, dev, torch
from tests.test_gpu_int8 import DT, tdt
from tests.test_mx_blocks import GRADIENTS, PRODUCTS

pytestmark = pytest.mark.gpu

GUARD = 4096


def codes(rows, K, seed):
    """Random codes, zeros past K (even), every scale 1."""
    T = torch()
    g = T.Generator(device=dev())
    g.manual_seed(seed)
    nb = -(-K // 32)
    c = T.randint(0, 256, (rows, 16 * nb), generator=g, device=dev(), dtype=T.uint8)
    c[:, K // 2:] = 0
    return c, T.full((rows, nb), 127, dtype=T.uint8, device=dev())


def values(c, s, K, t):
    return kb.dequantize_mxfp4(c, s, K, dtype=t)  # exact


class Space:
    """A workspace of exactly the size that is asked for, with guards behind it."""

    def __init__(self, need):
        self.buf = torch().full((need + GUARD,), 0xFF, dtype=torch().uint8, device=dev())
        self.ws = self.buf[:need]

    def check(self):
        assert (self.buf[-GUARD:] == 0xFF).all(), "written behind the workspace"


def same(got, want, what):
    assert torch().equal(got, want), (what, int((got != want).sum()))


@pytest.mark.parametrize("M,N,K", [p[:3] for p in PRODUCTS])
def test_products(M, N, K):
    # with all scales 1 sums are multiples of 1/4 below 36 K, at most 2^20: fp32 holds every partial sum in any order.  Some
    # rows and channels are at other powers of two: their sums scale as a whole.
    T, lib = torch(), kb.lib()
    t = tdt(DT[(M + N + K) % 3])
    a, w = codes(M, K, M), codes(N, K, N)
    a[1][::3], w[1][::5] = 125, 130
    bias = (T.randint(-64, 65, (N,), device=dev()) / 4).to(t)
    x = values(*a, K, T.float32)
    want = T.mm(x.double(), values(*w, K, T.float32).double().t().contiguous()).add_(bias.double())
    assert float(want.abs().max()) * 16 < 2 ** 24  # so is the sum with the bias, in multiples of 1/16
    want = want.to(t)
    case(f"linear mxfp4 of blocks {t} M={M} N={N} K={K}: codes")
    ws = Space(lib.linear_mxfp4_workspace_bytes(M, N, 32 * a[1].shape[1]))
    got = kb.linear_mxfp4(*a, *w, bias=bias, dtype=t, workspace=ws.ws)
    same(got, want, "codes")
    ws.check()
    got.zero_()
    case(f"linear mxfp4 of blocks {t} M={M} N={N} K={K}: values")
    ws = Space(lib.linear_mxfp4_dynamic_workspace_bytes(M, N, K))
    # values of a block's codes are codes of the scale that the quantizer takes, whatever it is
    kb.linear_mxfp4_dynamic(x.to(t), *w, bias=bias, out=got, workspace=ws.ws)
    same(got, want, "values")
    ws.check()
    same(kb.linear_mxfp4_dynamic(x.to(t), *w, bias=bias), want, "a workspace of its own")
    del a, w, x, want, got, ws
    T.cuda.empty_cache()


@pytest.mark.parametrize("M,N,K", [g[:3] for g in GRADIENTS])
def test_gradients(M, N, K):
    # values of codes with the scale 1, along rows and along columns: nothing is rounded
    T = torch()
    t = tdt(DT[(M + N) % 3])
    g, x, w = (values(*codes(r, d, r + 3 * d), d, t) for r, d in ((M, N), (M, K), (N, K)))
    g64 = g.double()
    dx = T.mm(g64, w.double()).to(t)
    dw = T.mm(g64.t().contiguous(), x.double())
    assert 144 * max(M, N) < 2 ** 24  # multiples of 1/4 below 36 M and 36 N
    case(f"linear mxfp4 backward of blocks {t} M={M} N={N} K={K}")
    ws = Space(kb.lib().linear_mxfp4_backward_workspace_bytes(M, N, K))
    for _ in range(2):  # the second in what the first left
        got = kb.linear_mxfp4_backward(g, x, w, workspace=ws.ws)
        same(got[0], dx, "dX")
        same(got[1], dw.float(), "dweight")
        same(got[2], g64.sum(0).float(), "dbias")
        ws.check()
    for i, only in enumerate(((True, False, False), (False, True, False), (False, False, True))):
        same(kb.linear_mxfp4_backward(g, x, w, *only)[i], got[i], f"alone {i}")
    T.cuda.empty_cache()

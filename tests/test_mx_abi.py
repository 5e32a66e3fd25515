"""Host-side checks of include/kbit_mx.h: exports, validation before any device
access, the binding's argument checks."""

import ctypes as ct
import os
import re
import subprocess

import pytest

kb = pytest.importorskip("blockwise_bit_codebook_amd")
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kbit_mx.h")
A = ct.c_void_p(0x10000)   # fake, never dereferenced device addresses
B8 = ct.c_void_p(0x20008)
B4 = ct.c_void_p(0x20004)
B2 = ct.c_void_p(0x20002)
B1 = ct.c_void_p(0x30001)
BIG = 1 << 50
FAR = 1 << 22


def test_header_compiles_as_c_and_cpp():
    for lang in ("c", "c++"):
        subprocess.run(["gcc", "-fsyntax-only", "-Wall", "-Werror", "-x", lang, HEADER], check=True)


def test_every_declared_symbol_is_exported_and_bound():
    out = subprocess.run(["gcc", "-E", "-P", "-x", "c", HEADER], capture_output=True, text=True, check=True).stdout
    names = sorted(set(re.findall(r"\b(?:int|int64_t)\s+(\w+)\s*\(", out)))
    assert len(names) == 5 + 3 * 8, names
    nm = subprocess.run(["nm", "-D", "--defined-only", os.path.join(ROOT, "blockwise_bit_codebook_amd", "libkbit.so")],
                        capture_output=True, text=True, check=True).stdout
    exported = set(l.split()[-1] for l in nm.splitlines() if " T " in l)
    assert not [n for n in names if n not in exported]
    from blockwise_bit_codebook_amd import _lib as L
    assert sorted(n for n, _ in L.MX_SIGNATURES) == names
    for n in ("quantize_mxfp4", "dequantize_mxfp4", "linear_mxfp4", "linear_mxfp4_dynamic", "linear_mxfp4_backward", "layer_norm",
              "layer_norm_backward"):
        assert n in kb.__all__ and callable(getattr(kb, n)) and getattr(kb, n).__doc__


def test_quantize_validation_codes():
    q = kb.lib().quantize_mxfp4_bf16
    assert q(None, 0, 100, 100, None, 64, None, 4, None) == 0            # no rows: no-op
    assert q(A, -1, 100, 100, A, 64, A, 4, None) == -1
    assert q(A, 2, 0, 100, A, 64, A, 4, None) == -1
    assert q(A, 2, (1 << 26) + 1, 1 << 27, A, 1 << 26, A, 1 << 22, None) == -1
    assert q(A, 2, 100, 99, A, 64, A, 4, None) == -1                     # rows overlap
    assert q(A, 2, 100, 100, A, 48, A, 4, None) == -1                    # no room for the last block
    assert q(A, 2, 100, 100, A, 64, A, 3, None) == -1
    assert q(A, 2, 100, 100, A, 72, A, 4, None) == -3                    # rows of codes not 16-byte aligned
    assert q(A, 2, 100, 100, B8, 64, A, 4, None) == -3
    assert q(B1, 2, 100, 100, A, 64, A, 4, None) == -3                   # an odd address of 16-bit elements
    assert q(A, 2, 100, 100, A, 64, None, 4, None) == -1 and q(A, 2, 100, 100, None, 64, A, 4, None) == -1
    assert q(None, 2, 100, 100, A, 64, A, 4, None) == -1
    assert kb.lib().quantize_mxfp4_fp32(B2, 2, 100, 100, A, 64, A, 4, None) == -3
    c = kb.lib().quantize_mxfp4_columns_fp16
    assert c(None, 100, 0, 0, None, 64, None, 4, None) == 0
    assert c(A, 0, 8, 8, A, 64, A, 4, None) == -1                        # columns of no values
    assert c(A, 100, 8, 7, A, 64, A, 4, None) == -1
    assert c(A, 100, 8, 8, A, 48, A, 4, None) == -1 and c(A, 100, 8, 8, A, 64, A, 3, None) == -1
    assert c(A, 100, -1, 8, A, 64, A, 4, None) == -1 and c(A, (1 << 26) + 1, 8, 8, A, 1 << 26, A, 1 << 22, None) == -1
    assert c(A, 100, (1 << 30) + 1, (1 << 30) + 1, A, 64, A, 4, None) == -1
    assert c(B1, 100, 8, 8, A, 64, A, 4, None) == -3 and c(A, 100, 8, 8, B4, 64, A, 4, None) == -3
    d = kb.lib().dequantize_mxfp4_bf16
    assert d(None, 64, None, 4, 0, 100, None, 100, None) == 0
    assert d(A, 64, A, 4, 2, 100, A, 99, None) == -1 and d(A, 48, A, 4, 2, 100, A, 100, None) == -1
    assert d(A, 64, A, 3, 2, 100, A, 100, None) == -1 and d(A, 64, None, 4, 2, 100, A, 100, None) == -1
    assert d(B8, 64, A, 4, 2, 100, A, 100, None) == -3 and d(A, 64, A, 4, 2, 100, B1, 100, None) == -3


def test_product_validation_codes():
    lib = kb.lib()

    def li(x=A, xs=A, M=4, K=100, ldx=64, ldxs=4, w=A, ws=A, N=64, ldw=64, ldws=4, bias=None, out=A, ldo=64, space=A, n=BIG):
        return lib.linear_mxfp4_fp16(x, xs, M, K, ldx, ldxs, w, ws, N, ldw, ldws, bias, out, ldo, space, n, None)
    assert li(M=0, x=None, xs=None, w=None, ws=None, out=None, space=None, n=0) == 0
    for kw in ({"out": None}, {"x": None}, {"xs": None}, {"w": None}, {"ws": None}, {"M": -1}, {"N": 0}, {"K": 0},
               {"K": (1 << 26) + 1, "M": 1, "N": 1}, {"ldx": 48}, {"ldxs": 3}, {"ldw": 48}, {"ldws": 3}, {"ldo": 63},
               {"ldx": FAR}, {"ldxs": FAR}, {"ldw": FAR}, {"ldws": FAR}):
        assert li(**kw) == -1, kw
    for kw in ({"x": B8}, {"w": B8}, {"ldx": 72}, {"ldw": 72}, {"out": B1}, {"bias": B1}, {"space": B4}):
        assert li(**kw) == -3, kw
    size = lib.linear_mxfp4_workspace_bytes
    assert size(0, 64, 64) >= 0 and size(-1, 64, 64) == -1 and size(4, 0, 64) == -1 and size(4, 64, 0) == -1
    assert size(4, 64, (1 << 26) + 1) == -1 and size(1 << 31, 64, 64) == -1

    dsize = lib.linear_mxfp4_dynamic_workspace_bytes
    assert dsize(4, 64, 0) == -1 and dsize(40, 64, 100) >= 40 * 64 + 160 + size(40, 64, 100)

    def dy(X=A, M=40, K=100, ldX=100, w=A, ws=A, N=64, ldw=64, ldws=4, bias=None, out=A, ldo=64, space=A, n=None):
        return lib.linear_mxfp4_dynamic_fp32(X, M, K, ldX, w, ws, N, ldw, ldws, bias, out, ldo, space,
                                             dsize(M, N, K) if n is None else n, None)
    assert dy(M=0, X=None, w=None, ws=None, out=None, space=None, n=0) == 0
    for kw in ({"X": None}, {"ldX": 99}, {"space": None}, {"n": 40 * 64}, {"n": -5}, {"w": None}, {"ldw": 48}, {"ldws": FAR},
               {"ldo": 63}, {"N": -1}):
        assert dy(**kw) == -1, kw
    for kw in ({"X": B2}, {"space": B4}, {"w": B8}, {"bias": B2}, {"out": B2}):
        assert dy(**kw) == -3, kw

    bsize = lib.linear_mxfp4_backward_workspace_bytes
    assert bsize(0, 64, 64) == 0 and bsize(-1, 64, 64) == -1 and bsize((1 << 26) + 1, 64, 64) == -1
    assert bsize(4, 0, 64) == -1 and bsize(4, 64, (1 << 26) + 1) == -1

    def back(g=A, ldg=64, X=A, ldx=100, W=A, ldw=100, M=40, N=64, K=100, dX=A, lddx=100, dW=A, lddw=100, db=A, space=A, n=None):
        return lib.linear_mxfp4_backward_bf16(g, ldg, X, ldx, W, ldw, M, N, K, dX, lddx, dW, lddw, db, space,
                                              bsize(M, N, K) if n is None else n, None)
    assert back(dX=None, dW=None, db=None, g=None, X=None, W=None, space=None) == 0
    assert back(M=0, dW=None, db=None, space=None) == 0
    for kw in ({"g": None}, {"X": None}, {"W": None}, {"ldg": 63}, {"ldx": 99}, {"ldw": 99}, {"lddx": 99}, {"lddw": 99},
               {"N": 0}, {"K": 0}, {"M": -1}, {"space": None}, {"n": 1000}, {"M": (1 << 26) + 1, "n": BIG},
               {"M": 1 << 24, "N": 1, "n": BIG}):  # columns of codes 8 MiB apart, out of the products' reach
        assert back(**kw) == -1, kw
    assert back(W=None, dX=None, n=1000) == -1 and back(X=None, dW=None, n=1000) == -1     # not missed, the workspace is
    for kw in ({"g": B1}, {"X": B1}, {"W": B1}, {"dX": B1}, {"dW": B2}, {"db": B2}, {"space": B8}):
        assert back(**kw) == -3, kw


def test_norm_validation_codes():
    lib = kb.lib()

    def norm(x=A, rows=4, d=100, ldx=100, w=A, b=None, fp32=0, eps=1e-5, out=A, ldo=100):
        return lib.layer_norm_bf16(x, rows, d, ldx, w, b, fp32, eps, out, ldo, None)
    assert norm(rows=0, x=None, w=None, out=None) == 0
    for kw in ({"x": None}, {"w": None}, {"out": None}, {"rows": -1}, {"d": 0}, {"d": (1 << 25) + 1, "rows": 1}, {"ldx": 99},
               {"ldo": 99}, {"eps": -1.0}, {"eps": float("nan")}, {"eps": float("inf")}):
        assert norm(**kw) == -1, kw
    for kw in ({"x": B1}, {"out": B1}, {"w": B1}, {"b": B1}, {"w": B2, "fp32": 1}, {"b": B2, "fp32": 1}):
        assert norm(**kw) == -3, kw
    size = lib.layer_norm_backward_workspace_bytes
    assert size(0, 100) == 0 and size(-1, 100) == -1 and size(4, 0) == -1 and size(4, (1 << 25) + 1) == -1
    assert size(1 << 31, 100) == -1

    def back(g=A, ldg=100, x=A, ldx=100, rows=4, d=100, w=A, fp32=0, eps=1e-5, dx=A, lddx=100, dw=A, db=A, space=A, n=None):
        return lib.layer_norm_backward_bf16(g, ldg, x, ldx, rows, d, w, fp32, eps, dx, lddx, dw, db, space,
                                            size(rows, d) if n is None else n, None)
    for kw in ({"g": None}, {"x": None}, {"w": None}, {"dx": None}, {"dw": None}, {"db": None}, {"space": None}, {"n": 100},
               {"ldg": 99}, {"ldx": 99}, {"lddx": 99}, {"eps": -1.0}, {"d": 0}, {"rows": -1, "n": BIG}):
        assert back(**kw) == -1, kw
    for kw in ({"g": B1}, {"x": B1}, {"dx": B1}, {"w": B2, "fp32": 1}, {"dw": B2}, {"db": B2}, {"space": B8}):
        assert back(**kw) == -3, kw


def bad(exc, match, fn, *a, **kw):
    with pytest.raises(exc, match=match):
        fn(*a, **kw)


def test_binding_refuses_on_the_host():
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    x = torch.zeros(4, 64, dtype=bf16)
    codes, scales = torch.zeros(4, 32, dtype=u8), torch.zeros(4, 2, dtype=u8)
    bad(TypeError, "X must be", kb.quantize_mxfp4, x[0])
    bad(TypeError, "X must be", kb.quantize_mxfp4, x.double())
    bad(TypeError, "X: expected a tensor", kb.quantize_mxfp4, None)
    bad(ValueError, "live on the GPU", kb.quantize_mxfp4, x)
    bad(ValueError, "live on the GPU", kb.dequantize_mxfp4, codes, scales, 64)
    bad(ValueError, "d must be between", kb.dequantize_mxfp4, codes, scales, 0)
    bad(ValueError, "d must be between", kb.dequantize_mxfp4, codes, scales, 1 << 27)
    bad(TypeError, "d must be an integer", kb.dequantize_mxfp4, codes, scales, "64")
    bad(TypeError, "dtype must be", kb.dequantize_mxfp4, codes, scales, 64, dtype=7)
    bad(TypeError, "unsupported element dtype", kb.dequantize_mxfp4, codes, scales, 64, dtype=torch.int8)
    bad(TypeError, "codes", kb.dequantize_mxfp4, x, scales, 64)
    bad(TypeError, "codes must be", kb.linear_mxfp4, x, scales, codes, scales)
    bad(ValueError, "live on the GPU", kb.linear_mxfp4, codes, scales, codes, scales)
    bad(TypeError, "X", kb.linear_mxfp4_dynamic, codes, codes, scales)
    bad(TypeError, "X: expected a tensor", kb.linear_mxfp4_dynamic, None, codes, scales)
    bad(ValueError, "live on the GPU", kb.linear_mxfp4_dynamic, x, codes, scales)
    bad(ValueError, "live on the GPU", kb.linear_mxfp4_backward, x, x, x)
    bad(TypeError, "dout: expected a tensor", kb.linear_mxfp4_backward, None, x, x)
    bad(ValueError, "live on the GPU", kb.layer_norm, x, x[0])
    bad(TypeError, "x must be", kb.layer_norm, x[0], x[0])
    bad(ValueError, "live on the GPU", kb.layer_norm_backward, x, x, x[0])


def test_star_import():
    names = {}
    exec("from blockwise_bit_codebook_amd import *", names)
    for n in ("quantize_mxfp4", "linear_mxfp4_dynamic", "linear_mxfp4_backward", "layer_norm", "layer_norm_backward"):
        assert callable(names[n])

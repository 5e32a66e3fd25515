"""Host-side checks of the operators around a quantized layer: exports of
include/kbit_layer.h, validation before any device access, the binding's
argument checks, and the host-computed frequencies."""

import ctypes as ct
import os
import re
import subprocess

import numpy as np
import pytest

from oracle import layer

kb = pytest.importorskip("blockwise_bit_codebook_amd")
torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kbit_layer.h")
A = ct.c_void_p(0x10000)   # fake, never dereferenced device addresses
B4 = ct.c_void_p(0x20004)
B1 = ct.c_void_p(0x30001)


def test_header_compiles_as_c_and_cpp():
    for lang in ("c", "c++"):
        subprocess.run(["gcc", "-fsyntax-only", "-Wall", "-Werror", "-x", lang, HEADER], check=True)


def test_every_declared_symbol_is_exported_and_bound():
    out = subprocess.run(["gcc", "-E", "-P", "-x", "c", HEADER], capture_output=True, text=True, check=True).stdout
    names = sorted(set(re.findall(r"\b(?:int|int64_t)\s+(\w+)\s*\(", out)))
    assert len(names) == 6 + 3 * 7, names
    nm = subprocess.run(["nm", "-D", "--defined-only", os.path.join(ROOT, "blockwise_bit_codebook_amd", "libkbit.so")],
                        capture_output=True, text=True, check=True).stdout
    exported = set(l.split()[-1] for l in nm.splitlines() if " T " in l)
    assert not [n for n in names if n not in exported]
    from blockwise_bit_codebook_amd import _lib as L
    assert sorted(n for n, _ in L.LAYER_SIGNATURES) == names
    for n in ("quantize_rows_int8", "linear_int8", "linear_int8_dynamic", "rope_frequencies", "rope_table", "rope",
              "qk_norm_rope", "qk_norm_rope_backward", "append_kv_paged"):
        assert n in kb.__all__ and callable(getattr(kb, n))


def test_int8_validation_codes():
    lib = kb.lib()
    q = lib.quantize_rows_int8_bf16
    assert q(None, 0, 100, 100, None, 112, None, None) == 0             # no rows: no-op
    assert q(A, -1, 100, 100, A, 112, A, None) == -1
    assert q(A, 2, 0, 100, A, 112, A, None) == -1                       # no columns
    assert q(A, 2, 100, 99, A, 112, A, None) == -1                      # rows overlap
    assert q(A, 2, 100, 100, A, 111, A, None) == -1                     # no room for the padding
    assert q(A, 2, 100, 100, A, 120, A, None) == -3                     # rows of codes not 16-byte aligned
    assert q(A, 2, 100, 100, B4, 112, A, None) == -3
    assert q(B1, 2, 100, 100, A, 112, A, None) == -3                    # an odd address of 16-bit elements
    assert q(A, 2, 100, 100, A, 112, None, None) == -1
    li = lib.linear_int8_fp16
    ws = lib.linear_int8_workspace_bytes(4, 64, 100)
    assert ws >= 0
    assert lib.linear_int8_workspace_bytes(4, 64, 131072) == -1         # the sum could leave int32
    assert lib.linear_int8_workspace_bytes(-1, 64, 64) == -1
    assert lib.linear_int8_dynamic_workspace_bytes(4, 64, 100) >= 4 * 112 + 16 + ws
    big = 1 << 40
    assert li(None, None, 0, 100, 100, None, None, 64, 100, None, None, 64, None, 0, None) == 0
    assert li(A, A, 4, 100, 100, A, A, 64, 100, None, None, 64, A, big, None) == -1       # no output
    assert li(A, None, 4, 100, 100, A, A, 64, 100, None, A, 64, A, big, None) == -1       # no scale
    assert li(A, A, 4, 131072, 131072, A, A, 64, 131072, None, A, 64, A, big, None) == -1
    assert li(A, A, 4, 100, 99, A, A, 64, 100, None, A, 64, A, big, None) == -1           # rows overlap
    assert li(A, A, 4, 100, 100, A, A, 64, 99, None, A, 64, A, big, None) == -1
    assert li(A, A, 4, 100, 100, A, A, 64, 100, None, A, 63, A, big, None) == -1
    assert li(A, B1, 4, 100, 100, A, A, 64, 100, None, A, 64, A, big, None) == -3
    assert li(A, A, 4, 100, 100, A, A, 64, 100, B1, A, 64, A, big, None) == -3
    dy = lib.linear_int8_dynamic_fp32
    need = lib.linear_int8_dynamic_workspace_bytes(4, 64, 100)
    assert dy(None, 0, 100, 100, None, None, 64, 100, None, None, 64, None, 0, None) == 0
    fused = lib.linear_int8_dynamic_fused
    assert fused(1, 4096, 4096, 4096) == 1 and fused(1, 4096, 4096, 4100) == 0       # unaligned rows of weights
    assert fused(9, 4096, 64, 64) == 0 and fused(0, 64, 64, 64) == 0 and fused(1, 64, 32768, 32768) == 0
    assert dy(A, 4, 100, 100, A, A, 64, 100, None, A, 64, A, need - 1, None) == -1
    assert dy(A, 4, 100, 100, A, A, 64, 100, None, A, 64, None, need, None) == -1
    assert dy(A, 4, 100, 100, A, A, 64, 100, None, A, 64, B4, need, None) == -3
    assert dy(A, 4, 100, 99, A, A, 64, 100, None, A, 64, A, need, None) == -1


def test_heads_validation_codes():
    lib = kb.lib()

    def rope(x=A, out=A, batch=1, tokens=4, heads=2, dim=64, pos=A, nbytes=8, table=A, rot=64, max_pos=16, layout=0):
        return lib.rope_bf16(x, 512, 128, 64, out, 512, 128, 64, batch, tokens, heads, dim, pos, nbytes, table, rot,
                             max_pos, layout, 0, None)
    assert rope(x=None, out=None, tokens=0, pos=None, table=None) == 0
    assert rope(dim=1025) == -1 and rope(dim=0) == -1 and rope(heads=0) == -1 and rope(tokens=-1) == -1
    assert rope(rot=63) == -1 and rope(rot=66) == -1 and rope(rot=0) == -1 and rope(max_pos=0) == -1
    assert rope(layout=2) == -1 and rope(nbytes=2) == -1
    assert rope(tokens=1 << 31) == -1 and rope(tokens=1 << 30, heads=2) == -1     # rows past 31 bits
    assert rope(batch=70000, tokens=2) == -1                                        # separate batches: grid axis
    assert rope(x=None) == -1 and rope(pos=None) == -1 and rope(table=None) == -1
    assert rope(x=B1) == -3 and rope(table=B4) == -3 and rope(pos=B4) == -3

    def norm(q=A, qw=A, fp32=0, eps=1e-6, dim=64, kh=1):
        return lib.qk_norm_rope_bf16(q, 0, 128, 64, A, 0, 128, 64, A, 0, 128, 64, A, 0, 128, 64, 1, 4, 2, kh, dim, qw,
                                     A, fp32, eps, A, 8, A, 64, 16, 0, None)
    assert norm(eps=-1.0) == -1 and norm(eps=float("nan")) == -1 and norm(eps=float("inf")) == -1
    assert norm(qw=None) == -1 and norm(kh=0) == -1 and norm(q=B1) == -3 and norm(qw=ct.c_void_p(0x10002), fp32=1) == -3
    assert lib.qk_norm_rope_backward_workspace_bytes(0) == -1
    assert lib.qk_norm_rope_backward_workspace_bytes(1025) == -1
    need = lib.qk_norm_rope_backward_workspace_bytes(64)

    def back(ws=A, n=need, dqw=A):
        v = [A, 0, 128, 64]
        return lib.qk_norm_rope_backward_bf16(*(v * 6), 1, 4, 2, 1, 64, A, A, 0, dqw, A, 1e-6, A, 8, A, 64, 16, 0, ws, n,
                                              None)
    assert back(ws=None) == -1 and back(n=need - 1) == -1 and back(dqw=None) == -1 and back(ws=B4) == -3

    def app(k=A, tokens=4, slots=A, nbytes=8, pages=8, page=16, rot=64, pos=A, table=A, dv=64):
        return lib.append_kv_paged_bf16(k, 128, 64, A, 128, 64, tokens, 2, 64, dv, slots, nbytes, A, 2048, 128, 64, A,
                                        2048, 128, 64, pages, page, pos, 8, table, rot, 16, 0, None)
    assert app(tokens=0) == 0 and app(pages=0) == 0
    assert app(page=0) == -1 and app(pages=1 << 28, page=16) == -1 and app(nbytes=1) == -1 and app(dv=0) == -1
    assert app(slots=None) == -1 and app(table=None) == -1 and app(pos=None) == -1 and app(rot=3) == -1
    assert app(k=B1) == -3 and app(slots=B4) == -3
    tb = lib.rope_table
    assert tb(A, 63, 8, 1.0, A, None) == -1 and tb(A, 64, 0, 1.0, A, None) == -1 and tb(None, 64, 8, 1.0, A, None) == -1
    assert tb(B4, 64, 8, 1.0, A, None) == -3 and tb(A, 64, 8, float("inf"), A, None) == -1


@pytest.mark.parametrize("rot", [2, 6, 64, 128, 1024])
@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
def test_frequencies(rot, scaling):
    kw = {} if scaling is None else {"factor": 4.0}
    if scaling == "yarn":
        kw["original_length"] = 4096
    f, amp = kb.rope_frequencies(rot, base=500000.0, scaling=scaling, **kw)
    want, wamp = layer.frequencies(rot, 500000.0, scaling, **kw)
    # a handful of fp64 roundings, pow and exp of arguments up to ln(5e5) apart
    assert np.allclose(f, want, rtol=1e-13) and abs(amp - wamp) < 1e-15


def test_frequency_refusals():
    for kw in ({"scaling": "other"}, {"scaling": "linear", "factor": 0.5}, {"scaling": "yarn", "factor": 2.0},
               {"scaling": "yarn", "factor": 2.0, "original_length": 64, "fast_turns": 1.0}, {"base": 1.0}):
        with pytest.raises((ValueError, kb.KbitError)):
            kb.rope_frequencies(64, **kw)
    for rot in (0, 7, 1026):
        with pytest.raises(kb.KbitError):
            kb.rope_frequencies(rot)


def bad(exc, match, fn, *a, **kw):
    with pytest.raises(exc, match=match):
        fn(*a, **kw)


def test_binding_refuses_on_the_host():
    bf16, f32, i8 = torch.bfloat16, torch.float32, torch.int8
    x = torch.zeros(4, 32, dtype=bf16)
    bad(TypeError, "X must be", kb.quantize_rows_int8, x[0])
    bad(TypeError, "X must be", kb.quantize_rows_int8, x.double())
    bad(ValueError, "live on the GPU", kb.quantize_rows_int8, x)
    bad(TypeError, "codes must be", kb.linear_int8, x, None, None, None)
    bad(ValueError, "live on the GPU", kb.linear_int8, x.to(i8), torch.zeros(4), x.to(i8), torch.zeros(4))
    bad(TypeError, "X: expected a tensor", kb.linear_int8_dynamic, None, x.to(i8), torch.zeros(4))
    h = torch.zeros(4, 2, 32, dtype=bf16)
    t = torch.zeros(8, 32)
    pos = torch.zeros(4, dtype=torch.int64)
    bad(ValueError, "live on the GPU", kb.rope, h, pos, t)
    bad(ValueError, "tokens, heads, dim", kb.rope, h[0], pos, t)
    bad(TypeError, "element type", kb.rope, h.double(), pos, t)
    bad(ValueError, "live on the GPU", kb.qk_norm_rope, h, h, t[0], t[0], pos, t)
    bad(ValueError, "live on the GPU", kb.append_kv_paged, h, h, pos, h[None], h[None])

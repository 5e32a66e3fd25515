"""Which way the layer operators' entry points send a call, seen on the host:
csrc/layer_api.cpp is linked with launchers that record their arguments
(tests/host/layer_stub.cpp)."""

import ctypes as ct
import os
import subprocess

import pytest

kb = pytest.importorskip("blockwise_bit_codebook_amd")
pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "blockwise_bit_codebook_amd", "csrc")
A = ct.c_void_p(0x10000)   # fake, never dereferenced addresses
B4 = ct.c_void_p(0x20004)


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("stub") / "layer_stub.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(CSRC, "layer_api.cpp"), os.path.join(ROOT, "tests", "host", "layer_stub.cpp"), "-o", so],
                   check=True)
    from blockwise_bit_codebook_amd import _lib as L
    lib = ct.CDLL(so)
    for name, args in L.LAYER_SIGNATURES:
        getattr(lib, name).argtypes = args
    return lib


def product(stub, x=A, M=1, K=100, ldx=100, w=A, N=64, ldw=112):
    before = stub.stub_product_launches()
    assert stub.linear_int8_bf16(x, A, M, K, ldx, w, A, N, ldw, None, A, N, None, 0, None) == 0
    assert stub.stub_product_launches() == before + 1
    return stub.stub_product_on_fast_path()


def test_a_single_row_needs_no_distance_to_the_next(stub):
    # a row of codes that starts at 16 bytes is aligned, whatever its depth
    assert product(stub) == 1
    assert product(stub, K=3000, ldx=3000, ldw=3008) == 1
    assert product(stub, M=7, ldx=112, N=1, ldw=100) == 1
    assert product(stub, M=1, ldx=99999, N=1, ldw=101) == 1
    # two rows do, and a start at 4 bytes is not at 16
    assert product(stub, M=2) == 0 and product(stub, M=2, ldx=112) == 1
    assert product(stub, ldw=100) == 0
    assert product(stub, x=B4) == 0 and product(stub, w=B4) == 0


def test_tokens_on_a_single_channel_need_no_distance_to_the_next():
    fused = kb.lib().linear_int8_dynamic_fused
    assert fused(1, 1, 100, 100) == 1 and fused(1, 1, 100, 1 << 22) == 1
    assert fused(1, 2, 100, 100) == 0 and fused(1, 2, 100, 1 << 22) == 0


def test_a_workspace_for_the_largest_batch_serves_every_smaller_one(stub):
    # on 256 compute units a product of 128 rows puts its depth in parts, one of 256 does not
    size, dynamic = stub.linear_int8_workspace_bytes, stub.linear_int8_dynamic_workspace_bytes
    size.restype = dynamic.restype = stub.stub_product_workspace.restype = ct.c_int64
    stub.stub_product_workspace.argtypes = [ct.c_int64, ct.c_int, ct.c_int]
    for N, K in ((4096, 11008), (4096, 4096), (1000, 3000), (130, 16384), (20000, 8192), (40000, 4096), (130, 256), (127, 9999),
                 ((1 << 20) + 4096, 11008)):
        before = before_dynamic = 0
        for M in sorted([*range(1, 700, 7), 128, 256, 512, 1024, 2048, 4096, 8192, 32768, 32769, 33000, 65536, 100000]):
            now, now_dynamic = size(M, N, K), dynamic(M, N, K)
            assert now >= before and now_dynamic >= before_dynamic, (M, N, K)
            assert now <= 256 * 2 * 65536
            # what the call itself asks for is no more than that
            assert stub.linear_int8_bf16(A, A, M, K, 1 << 15, A, A, N, 1 << 15, None, A, N, A, now, None) == 0, (M, N, K)
            assert stub.linear_int8_dynamic_bf16(A, M, K, K, A, A, N, 1 << 15, None, A, N, A, now_dynamic, None) == 0
            before, before_dynamic = now, now_dynamic
    needs = [stub.stub_product_workspace(M, 4096, 11008) for M in (64, 128, 256, 512, 2048)]
    assert 0 < needs[1] < needs[3] and needs[0] == needs[2] == needs[4] == 0


def test_the_longest_row_of_codes(stub):
    # the kernels round a row's length up to 16 in 32 bits
    def rows(d):
        return stub.quantize_rows_int8_bf16(A, 1, d, d, A, 1 << 31, A, None)
    assert rows((1 << 31) - 16) == 0
    assert [rows((1 << 31) - k) for k in (15, 2, 1)] == [-1, -1, -1]

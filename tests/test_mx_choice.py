"""Which kernel the MXFP4 product's rule picks on 256 compute units, for every
shape that tests/test_gpu_mx_choice.py runs to reach that kernel's loops, and
what the entry points of include/kbit_mx.h launch: csrc/mx_api.cpp is linked
with launchers that count (tests/host/mx_stub.cpp)."""

import ctypes as ct
import os
import random
import subprocess

import pytest

kb = pytest.importorskip("blockwise_bit_codebook_amd")
pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "blockwise_bit_codebook_amd", "csrc")
A = ct.c_void_p(0x10000)   # fake, never dereferenced addresses
BIG = 1 << 50

# Pieces of few rows, in 16 x 16: the waves that split the depth (up to a row of 4096 bytes of codes, beyond).
WAVES = {(1, 1): (4, 8), (1, 2): (8,), (1, 3): (8,), (1, 4): (7,), (2, 2): (8,), (2, 4): (6,), (3, 2): (6,), (3, 4): (5,),
         (4, 4): (4,), (5, 3): (4,), (5, 4): (4,)}

# (pieces, M, N, K): every wave has more than two steps, not all as many; the last step whole and partial.
FEW = [((1, 1), 1, 1, 2273), ((1, 1), 9, 40, 2305), ((1, 1), 1, 1, 8419), ((1, 1), 7, 33, 8451), ((1, 2), 1, 4192, 4322),
       ((1, 2), 1, 4219, 4355), ((1, 3), 1, 8854, 4352), ((1, 3), 1, 8346, 4466), ((1, 4), 1, 12490, 3821),
       ((1, 4), 1, 12350, 3877), ((2, 2), 4151, 1, 4588), ((2, 2), 4181, 1, 4383), ((2, 4), 18, 8660, 3324),
       ((2, 4), 17, 8351, 3337), ((3, 2), 8203, 1, 3319), ((3, 2), 8193, 1, 3358), ((3, 4), 8514, 34, 2789),
       ((3, 4), 8213, 35, 2860), ((4, 4), 7007, 103, 2291), ((4, 4), 6953, 98, 2353), ((5, 3), 6245, 72, 2538),
       ((5, 3), 6313, 66, 2314), ((5, 4), 9338, 107, 2280), ((5, 4), 8359, 98, 2494)]

# (rows of the tile, stages of the ring, M, N, K): every count of steps modulo the stages, the last one whole and partial.
RING = [(32, 2, 34, 16947, 2020), (32, 2, 33, 17984, 2126), (32, 2, 34, 17236, 2295), (32, 2, 33, 16443, 2437),
        (32, 4, 82, 2040, 2032), (32, 4, 33, 5451, 2268), (32, 4, 75, 2763, 2274), (32, 4, 49, 4123, 2400),
        (32, 4, 1709, 129, 2530), (32, 4, 51, 4130, 2590), (32, 4, 50, 4416, 2789), (32, 4, 52, 4116, 2981),
        (64, 2, 8640, 136, 2028), (64, 2, 66, 16409, 2146), (64, 2, 68, 16695, 2277), (64, 2, 66, 16539, 2365),
        (64, 4, 4338, 131, 2019), (64, 4, 4407, 131, 2130), (64, 4, 4254, 139, 2279), (64, 4, 4249, 131, 2337),
        (64, 4, 4461, 145, 2555), (64, 4, 4269, 135, 2686), (64, 4, 2788, 259, 2816), (64, 4, 4206, 137, 2818),
        (128, 2, 197, 16769, 2040), (128, 2, 194, 16396, 2131), (128, 2, 641, 5399, 2291), (128, 2, 197, 16817, 2373),
        (128, 4, 5717, 265, 2045), (128, 4, 8334, 133, 2088), (128, 4, 6255, 257, 2287), (128, 4, 8259, 130, 2316),
        (128, 4, 9044, 147, 2548), (128, 4, 8208, 134, 2589), (128, 4, 5934, 261, 2808), (128, 4, 8269, 141, 2858)]

# Tiles of 256: pairs of steps alone, a step beyond them, part of one; channels in whole 16-byte pieces and not.
LARGE = [(5831, 2049, 1508), (1859, 7104, 1521), (6530, 1793, 1253), (1737, 6944, 1278), (781, 14278, 1029), (778, 14744, 1030)]

# (parts of the depth, stages, M, N, K)
PARTS = [(2, 2, 8297, 138, 12274), (2, 4, 1005, 1301, 16218), (3, 2, 8488, 129, 13797), (3, 4, 4195, 136, 18170),
         (4, 2, 4555, 146, 20426), (4, 4, 150, 2060, 18216), (7, 2, 149, 2365, 21353), (7, 4, 852, 133, 21455),
         (8, 2, 148, 2079, 18796), (8, 4, 210, 290, 27706)]


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("mx_stub") / "mx_stub.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(CSRC, "mx_api.cpp"), os.path.join(ROOT, "tests", "host", "mx_stub.cpp"), "-o", so], check=True)
    from blockwise_bit_codebook_amd import _lib as L
    lib = ct.CDLL(so)
    for name, args in L.MX_SIGNATURES:
        getattr(lib, name).argtypes = args
        if name.endswith("_bytes"):
            getattr(lib, name).restype = ct.c_int64
    lib.stub_mx_form.argtypes = [ct.c_int64, ct.c_int, ct.c_int, ct.c_int64, ct.c_void_p]
    lib.stub_mx_workspace.argtypes = [ct.c_int64, ct.c_int, ct.c_int]
    lib.stub_mx_workspace.restype = ct.c_int64
    return lib


def form(stub, M, N, K, cus=256):
    v = (ct.c_int * 4)()
    stub.stub_mx_form(M, N, K, cus, v)
    return v[0], (v[1], v[2]), v[3]


def row_bytes(K):
    return -(-K // 32) * 16


def tiles(M, N, bm, bn):
    return -(-M // bm) * -(-N // bn)


@pytest.mark.parametrize("pieces,M,N,K", FEW)
def test_few_rows(stub, pieces, M, N, K):
    assert form(stub, M, N, K) == (0, pieces, 1)
    waves = WAVES[pieces][-1 if row_bytes(K) > 4096 else 0]
    steps = row_bytes(K) // 128
    assert steps > 2 * waves and steps % waves != 0


@pytest.mark.parametrize("bm,stages,M,N,K", RING)
def test_ring(stub, bm, stages, M, N, K):
    assert form(stub, M, N, K) == (bm, (0, 0), 1)
    assert (tiles(M, N, bm, 128) <= 256) == (stages == 4) and row_bytes(K) // 128 >= 7


@pytest.mark.parametrize("M,N,K", LARGE)
def test_large(stub, M, N, K):
    assert form(stub, M, N, K) == (256, (0, 0), 1)


@pytest.mark.parametrize("parts,stages,M,N,K", PARTS)
def test_parts(stub, parts, stages, M, N, K):
    assert form(stub, M, N, K) == (128, (0, 0), parts)
    assert (tiles(M, N, 128, 128) * parts <= 256) == (stages == 4)


def test_every_form_is_listed(stub):
    for pieces in WAVES:
        assert {row_bytes(K) % 128 != 0 for p, _, _, K in FEW if p == pieces} == {False, True}
    for bm in (32, 64, 128):
        for stages in (2, 4):
            seen = {(row_bytes(K) // 128 % stages, row_bytes(K) % 128 != 0) for b, s, _, _, K in RING if (b, s) == (bm, stages)}
            assert len(seen) == 2 * stages
    assert {(row_bytes(K) % 256 + 127) // 128 + (row_bytes(K) % 128 != 0) for _, _, K in LARGE} >= {0, 1}
    # nothing else comes up
    listed = {(0, p, 1) for p in WAVES} | {(bm, (0, 0), 1) for bm in (32, 64, 128, 256)} | {(128, (0, 0), p) for p, *_ in PARTS}
    rng = random.Random(5)
    for _ in range(20000):
        M, N, K = (int(2 ** rng.uniform(lo, hi)) for lo, hi in ((0, 15), (0, 20), (0, 26)))
        bm, pieces, parts = form(stub, M, N, K)
        assert (bm, pieces, parts) in listed or (bm == 128 and 2 <= parts <= 8), (M, N, K, bm, pieces, parts)


def test_a_workspace_for_the_largest_batch_serves_every_smaller_one(stub):
    rng = random.Random(6)
    size, dynamic = stub.linear_mxfp4_workspace_bytes, stub.linear_mxfp4_dynamic_workspace_bytes
    back, norm = stub.linear_mxfp4_backward_workspace_bytes, stub.layer_norm_backward_workspace_bytes
    for _ in range(3000):
        M, N, K = (int(2 ** rng.uniform(lo, hi)) for lo, hi in ((0, 17), (0, 15), (0, 15)))
        less = rng.randint(1, M)
        assert stub.stub_mx_workspace(less, N, K) <= size(less, N, K) <= size(M, N, K)
        assert dynamic(less, N, K) <= dynamic(M, N, K)
        assert back(less, N, K) <= back(M, N, K)
        assert norm(less, N) <= norm(M, N)
    # as the entry points see it
    for parts, _, M, N, K in PARTS:
        need = size(4 * M, N, K)
        assert stub.linear_mxfp4_bf16(A, A, M, K, row_bytes(K), row_bytes(K), A, A, N, row_bytes(K), row_bytes(K), None, A, N, A,
                                      need, None) == 0
        assert stub.stub_mx_workspace(M, N, K) >= parts * M * N * 4
        assert stub.linear_mxfp4_bf16(A, A, M, K, row_bytes(K), row_bytes(K), A, A, N, row_bytes(K), row_bytes(K), None, A, N, A,
                                      parts * M * N * 4 - 1, None) == -1


def counts(stub, fn):
    a, b = (ct.c_int * 5)(), (ct.c_int * 5)()
    stub.stub_counts(a)
    assert fn() == 0
    stub.stub_counts(b)
    return [y - x for x, y in zip(a, b)]   # launches: all, products, of tokens, over rows; matrices over columns


def test_launches(stub):
    def dynamic(M, N, K, ldw=None, ldws=None):
        return counts(stub, lambda: stub.linear_mxfp4_dynamic_bf16(
            A, M, K, K, A, A, N, row_bytes(K) if ldw is None else ldw, -(-K // 32) if ldws is None else ldws, None, A, N, A, BIG,
            None))
    assert dynamic(1, 4096, 4096) == [1, 0, 1, 0, 0]
    assert dynamic(8, 640, 2048) == [1, 0, 1, 0, 0] and dynamic(4, 640, 4096) == [1, 0, 1, 0, 0]
    assert dynamic(5, 640, 4096) == [2, 1, 0, 1, 0]  # 5 rows of 8 pieces of 512 values: more than 32
    assert dynamic(9, 640, 4096) == [2, 1, 0, 1, 0]
    assert dynamic(1, 640, 32768) == [2, 1, 0, 1, 0] and dynamic(8, 640, 8192) == [2, 1, 0, 1, 0]
    assert dynamic(4096, 4096, 4096) == [2, 1, 0, 1, 0] and stub.stub_paired() == 1   # its own scales, not the caller's
    assert dynamic(600, 600, 600) == [2, 1, 0, 1, 0] and stub.stub_paired() == 0
    assert dynamic(40000, 4096, 4096) == [2, 1, 0, 1, 0] and stub.stub_paired() == 0  # more than one block of rows

    def back(M, N, K, dx=A, dw=A, db=A):
        return counts(stub, lambda: stub.linear_mxfp4_backward_bf16(A, N, A, K, A, K, M, N, K, dx, K, dw, K, db, A, BIG, None))
    assert back(64, 96, 128) == [4, 2, 0, 0, 3]           # dout both ways and its sums in one reading, three matrices in one launch
    assert back(64, 96, 128, dw=None) == [3, 1, 0, 0, 2]
    assert back(64, 96, 128, dw=None, db=None) == [3, 1, 0, 1, 1]
    assert back(64, 96, 128, dx=None, db=None) == [2, 1, 0, 0, 2]
    assert back(64, 96, 128, dx=None, dw=None) == [2, 0, 0, 0, 1]
    assert back(64, 96, 128, dx=None, dw=None, db=None) == [0] * 5
    assert back(0, 96, 128) == [2, 0, 0, 0, 0]            # zeros
    assert back(0, 96, 128, dw=None, db=None) == [0] * 5
    assert back(4096, 4096, 4096, dw=None) == [3, 1, 0, 0, 2] and stub.stub_paired() == 3


def test_tokens_that_fit():
    fused = kb.lib().linear_mxfp4_dynamic_fused
    assert fused(1, 4096, 4096, 2048, 128) == 1 and fused(4, 4096, 4096, 2048, 128) == 1
    assert fused(5, 4096, 4096, 2048, 128) == 0 and fused(8, 4096, 2048, 1024, 64) == 1  # 32 pieces of 512 values
    assert fused(9, 4096, 64, 32, 2) == 0 and fused(0, 64, 64, 32, 2) == 0 and fused(1, 64, 32768, 16384, 1024) == 0
    assert fused(1, 2, 100, 1 << 22, 4) == 0 and fused(1, 2, 100, 64, 1 << 22) == 0 and fused(1, 1, 100, 1 << 22, 1 << 22) == 1
    assert fused(1, (1 << 20) + 1, 100, 64, 4) == 0

"""What the entry points of include/kbit_mx.h write of their workspaces: csrc/mx_api.cpp
is linked with launchers that record it (tests/host/mx_space_stub.cpp)."""

import ctypes as ct
import itertools
import os
import random
import subprocess

import pytest

pytest.importorskip("blockwise_bit_codebook_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "blockwise_bit_codebook_amd", "csrc")
A = 0x10000        # fake, never dereferenced addresses
SPACE = 1 << 40
GRADIENTS = [c for c in itertools.product((0, 1), repeat=3) if any(c)]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("mx_space") / "mx_space.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(CSRC, "mx_api.cpp"), os.path.join(ROOT, "tests", "host", "mx_space_stub.cpp"), "-o", so], check=True)
    from blockwise_bit_codebook_amd import _lib as L
    lib = ct.CDLL(so)
    for name, args in L.MX_SIGNATURES:
        getattr(lib, name).argtypes = args
        if name.endswith("_bytes"):
            getattr(lib, name).restype = ct.c_int64
    lib.space_back.argtypes = [ct.c_int64] + [ct.c_int] * 5
    lib.space_back.restype = ct.c_int64
    lib.space_written.argtypes = [ct.c_void_p, ct.c_int]
    return lib


def written(lib):
    v = (ct.c_int64 * 32)()
    n = lib.space_written(v, 16)
    return [(v[2 * i], v[2 * i + 1]) for i in range(n)]


def back(lib, M, N, K, which, n):
    dX, dW, db = (A if w else None for w in which)
    return lib.linear_mxfp4_backward_bf16(A, N, A, K, A, K, M, N, K, dX, K, dW, K, db, SPACE, n, None)


def sizes(seed, count):
    rng = random.Random(seed)
    yield from ((1, 1, 1), (333, 1000, 1031), (8192, 4096, 4096), (8192, 11008, 4096), (33100, 520, 96))
    for _ in range(count):
        yield tuple(int(2 ** rng.uniform(0, hi)) for hi in (16, 14, 14))


def test_parts_of_the_backward_pass_are_inside_and_apart(lib):
    for M, N, K in sizes(1, 300):
        for which in GRADIENTS:
            need = lib.space_back(M, N, K, *which)
            assert back(lib, M, N, K, which, need - 1) == -1 and not written(lib)
            assert back(lib, M, N, K, which, need) == 0
            parts = sorted(written(lib))
            assert all(SPACE <= at and at + n <= SPACE + need for at, n in parts), (M, N, K, which)
            for (a, n), (b, _) in zip(parts, parts[1:]):  # the products' own, one after the other in one place, comes last
                assert a + n <= b or a == b == parts[-1][0], (M, N, K, which)


def test_a_gradient_takes_no_more_than_its_own_operands(lib):
    def rows(r, d):  # codes in whole cache lines, scales in whole pairs of steps
        blocks = -(-d // 32)
        return r * (-(-blocks // 8) * 128 + -(-blocks // 16) * 16)
    for M, N, K in sizes(2, 100):
        up = lambda n: -(-n // 128) * 128  # noqa: E731
        assert lib.space_back(M, N, K, 0, 0, 1) == up(4 * -(-M // 256) * N)
        for which, own in (((1, 0, 0), ((M, N), (K, N))), ((0, 1, 0), ((N, M), (K, M)))):
            least = sum(up(rows(*o)) for o in own)
            products = lib.space_back(M, N, K, *which) - least
            assert 0 <= products <= lib.linear_mxfp4_workspace_bytes(own[0][0], K, own[0][1])
    assert lib.space_back(8192, 11008, 4096, 0, 0, 1) < 2 << 20


def test_the_public_size_serves_every_choice_and_fewer_rows(lib):
    rng = random.Random(3)
    for M, N, K in sizes(4, 300):
        size = lib.linear_mxfp4_backward_workspace_bytes(M, N, K)
        for less in (M, rng.randint(1, M)):
            for which in GRADIENTS:
                assert lib.space_back(less, N, K, *which) <= size, (less, M, N, K, which)


def test_the_dynamic_product_stays_inside(lib):
    for M, N, K in sizes(5, 300):
        row = -(-K // 32) * 16
        size = lib.linear_mxfp4_dynamic_workspace_bytes(M, N, K)
        assert lib.linear_mxfp4_dynamic_bf16(A, M, K, K, A, A, N, row, -(-K // 32), None, A, N, SPACE, size, None) == 0
        parts = sorted(written(lib))
        assert all(SPACE <= at and at + n <= SPACE + size for at, n in parts), (M, N, K)
        assert all(a + n <= b for (a, n), (b, _) in zip(parts, parts[1:])), (M, N, K)

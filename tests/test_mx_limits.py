"""The limits that include/kbit_mx.h states for the MXFP4 products and gradients,
on either side of them, over launchers that only count; the sizes of workspaces
know them too."""

import ctypes as ct

import pytest

pytest.importorskip("blockwise_bit_codebook_amd")
pytest.importorskip("torch")

from tests.test_mx_choice import row_bytes, stub  # noqa: E402, F401

A = ct.c_void_p(0x10000)   # fake, never dereferenced addresses
BIG = 1 << 60
MOST = (1 << 23) - 256     # values of rows in a workspace
LONGEST = 1 << 26


def linear(lib, M, N, K):
    row, scales = row_bytes(K), -(-K // 32)
    return lib.linear_mxfp4_bf16(A, A, M, K, row, scales, A, A, N, row, scales, None, A, N, A, BIG, None)


def dynamic(lib, M, N, K):
    return lib.linear_mxfp4_dynamic_bf16(A, M, K, K, A, A, N, row_bytes(K), -(-K // 32), None, A, N, A, BIG, None)


def back(lib, M, N, K, dX=A, dW=A, db=A):
    return lib.linear_mxfp4_backward_bf16(A, N, A, K, A, K, M, N, K, dX, K, dW, K, db, A, BIG, None)


def test_products_of_codes(stub):  # noqa: F811
    size = stub.linear_mxfp4_workspace_bytes
    near, far = (1 << 23) - 32, (1 << 23) - 31  # codes of a row: 2^22 - 16 bytes, 2^22
    for M, N in ((2, 1), (1, 2), (300, 300)):
        assert linear(stub, M, N, near) == 0 and size(M, N, near) >= 0
        assert linear(stub, M, N, far) == -1 and size(M, N, far) == -1
    for K in (far, LONGEST):
        assert linear(stub, 1, 1, K) == 0 and size(1, 1, K) >= 0
    assert linear(stub, 1, 1, LONGEST + 1) == -1 and size(1, 1, LONGEST + 1) == -1


def test_products_of_values(stub):  # noqa: F811
    size, fused = stub.linear_mxfp4_dynamic_workspace_bytes, stub.linear_mxfp4_dynamic_fused
    for M, N in ((2, 1), (9, 64)):
        assert dynamic(stub, M, N, MOST) == 0 and size(M, N, MOST) > 0
        assert dynamic(stub, M, N, MOST + 1) == -1 and size(M, N, MOST + 1) == -1
    assert dynamic(stub, 1, 2, (1 << 23) - 32) == 0 and size(1, 2, (1 << 23) - 32) > 0   # the weight's own distance
    assert dynamic(stub, 1, 2, (1 << 23) - 31) == -1 and size(1, 2, (1 << 23) - 31) == -1
    assert dynamic(stub, 1, 1, LONGEST) == 0 and size(1, 1, LONGEST) > 0
    assert not fused(9, 64, MOST + 1, row_bytes(MOST + 1), 1 << 19)


def test_gradients(stub):  # noqa: F811
    size = stub.linear_mxfp4_backward_workspace_bytes
    # dX sums over N
    assert back(stub, 2, MOST, 3, dW=None) == 0 and back(stub, 2, MOST + 1, 3, dW=None) == -1
    assert back(stub, 1, MOST + 1, 2, dW=None) == -1 and back(stub, 1, MOST + 1, 1, dW=None) == 0
    assert back(stub, 2, MOST + 1, 3, dX=None) == 0 and back(stub, 2, LONGEST, 3, dX=None, dW=None) == 0
    # dW over M
    assert back(stub, MOST, 3, 2, dX=None) == 0 and back(stub, MOST + 1, 3, 2, dX=None) == -1
    assert back(stub, MOST + 1, 1, 2, dX=None) == -1 and back(stub, MOST + 1, 1, 1, dX=None) == 0
    assert back(stub, MOST + 1, 3, 2, dW=None) == 0 and back(stub, LONGEST, 3, 2, dX=None, dW=None) == 0
    assert back(stub, 2, 3, LONGEST) == 0
    # a size for what some gradients take
    assert size(2, LONGEST, 3) > 0 and size(LONGEST, 3, 2) > 0 and size(2, 3, LONGEST) > 0
    for bad in ((LONGEST + 1, 3, 2), (2, LONGEST + 1, 3), (2, 3, LONGEST + 1)):
        assert size(*bad) == -1 and back(stub, *bad) == -1

"""Products of more than 32768 rows or 2^20 channels run block by block: which
kernel each block of the shapes of tests/test_gpu_mx_blocks.py reaches, on 256
compute units."""

import pytest

pytest.importorskip("blockwise_bit_codebook_amd")
pytest.importorskip("torch")

from tests.test_mx_choice import form, row_bytes, stub  # noqa: E402, F401

ROWS, CHANNELS = 1 << 15, 1 << 20

# (M, N, K, forms of the blocks: rows of the tile or pieces of few rows in 16 x 16, parts of the depth). One block leaves
# its scales in the order of pairs in the workspace or the sums of its parts, where the next one finds them.
PRODUCTS = [(32769, 512, 512, [256, (1, 1)]),
            (33100, 512, 520, [256, 32]),
            (33000, 1024, 2100, [256, (2, 2)]),
            (70000, 1000, 544, [256, 256, 128]),
            (32918, 2060, 18216, [256, (128, "parts", 4)]),
            (32978, 290, 27706, [128, (128, "parts", 8)]),
            (3, CHANNELS + 5, 96, [(1, 4), (1, 1)]),
            (260, CHANNELS + 130, 64, [128, 32]),
            (768, CHANNELS + 130, 800, [256, (1, 2)])]

# (M, N, K, forms of dX's blocks, forms of dweight's)
GRADIENTS = [(33100, 512, 512, [256, 32], [(128, "parts", 8)]),
             (32769, 2100, 1024, [256, (1, 1)], [(128, "parts", 3)]),
             (40000, 96, 200, [128, 32], [(1, 1)])]


def blocks(n, most):
    return [min(most, n - i) for i in range(0, n, most)]


def forms(stub, M, N, K):  # noqa: F811
    out = []
    for n in blocks(N, CHANNELS):
        for m in blocks(M, ROWS):
            bm, few, parts = form(stub, m, n, K)
            out.append(few if bm == 0 else (bm, "parts", parts) if parts > 1 else bm)
    return out


@pytest.mark.parametrize("M,N,K,want", PRODUCTS)
def test_products(stub, M, N, K, want):  # noqa: F811
    assert forms(stub, M, N, K) == want


@pytest.mark.parametrize("M,N,K,dx,dw", GRADIENTS)
def test_gradients(stub, M, N, K, dx, dw):  # noqa: F811
    assert forms(stub, M, K, N) == dx and forms(stub, N, K, M) == dw


def test_workspaces_hold_every_block(stub):  # noqa: F811
    for M, N, K, _ in PRODUCTS:
        size = stub.linear_mxfp4_workspace_bytes(M, N, K)
        for n in blocks(N, CHANNELS):
            for m in blocks(M, ROWS):
                assert stub.stub_mx_workspace(m, n, K) <= stub.stub_mx_workspace(M, N, K) <= size
    assert row_bytes(18216) == 9120  # the sums of parts of 150 x 2060 and the scales of 32768 + 2060 rows
    assert stub.stub_mx_workspace(32918, 2060, 18216) >= max(4 * 150 * 2060 * 4, (32768 + 2060) * 36 * 16)

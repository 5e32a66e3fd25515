"""Which kernel the int8 product's rule picks on 256 compute units, for every
shape that tests/test_gpu_int8_choice.py runs to reach that kernel's loops: a
change of the estimates cannot move one of them to another kernel unseen."""

import ctypes as ct

import pytest

from tests.test_layer_dispatch import stub  # noqa: F401  (fixture)

# Pieces of few rows, in 16 x 16: the waves that split the depth.
WAVES = {(1, 1): (4, 8), (1, 2): (8,), (1, 3): (8,), (1, 4): (7,), (2, 2): (8,), (2, 4): (6,), (3, 2): (6,), (3, 4): (5,),
         (4, 4): (4,), (5, 3): (4,), (5, 4): (4,), (7, 3): (4,), (8, 3): (3,)}

# (pieces, M, N, K): deep enough that every wave loads over a step it has read
# (more than two steps a wave), and not the same number of steps for all; the
# last step whole and partial.
FEW = [((1, 1), 2, 36, 1152), ((1, 1), 11, 300, 1158), ((1, 1), 7, 40, 4224), ((1, 1), 15, 50, 4255),
       ((1, 2), 2, 4175, 2176), ((1, 2), 92, 807, 4454), ((1, 3), 2, 8282, 2176), ((1, 3), 45, 2741, 4644),
       ((1, 4), 2, 12690, 1920), ((1, 4), 7, 15354, 8195), ((2, 2), 4420, 4, 2176), ((2, 2), 723, 293, 7131),
       ((2, 4), 17, 8458, 1792), ((2, 4), 687, 626, 3253), ((3, 2), 4121, 35, 1664), ((3, 2), 2263, 113, 4031),
       ((3, 4), 4400, 68, 1408), ((3, 4), 1379, 357, 2497), ((3, 4), 48, 11008, 4096), ((3, 4), 128, 4099, 4000),
       ((4, 4), 192, 4099, 3968), ((4, 4), 7631, 97, 1188), ((5, 3), 6203, 71, 1152), ((5, 3), 6390, 69, 1156),
       ((5, 4), 70, 12668, 1792), ((5, 4), 65, 13094, 1826), ((7, 3), 90, 8237, 2432), ((7, 3), 84, 10181, 2357),
       ((8, 3), 117, 8201, 2944), ((8, 3), 115, 9818, 2947)]

# (rows of the tile, M, N, K): several pairs of steps, and beyond them nothing, a
# partial step, a whole one, both.
TILES = [(32, 49, 4183, 768), (32, 33, 8429, 769), (32, 51, 4098, 896), (32, 33, 8463, 910),
         (64, 4344, 130, 768), (64, 7928, 129, 769), (64, 4667, 130, 896), (64, 101, 14723, 918),
         (128, 130, 14018, 768), (128, 132, 15047, 769), (128, 129, 13595, 896), (128, 129, 15191, 933)]

# Tiles of 256 rows whose workgroups do not stay: odd channels with nothing
# beyond the pairs of steps, then as above, with outputs of whole pieces too.
LARGE = [(646, 11252 + 1, 768), (538, 13071, 769), (656, 11137, 896), (541, 13123, 897), (2100, 4104, 640), (1100, 8200, 1000)]

# Workgroups that stay, more tiles than compute units and fewer.
STAY = [(8200, 2600, 512), (2700, 8200, 768), (7172, 1032, 768)]

# (parts of the depth, M, N, K)
PARTS = [(2, 6983, 138, 2874), (3, 208, 4237, 2295), (4, 171, 5815, 4096), (7, 237, 2062, 3506), (8, 1565, 236, 6046)]


def form(stub, M, N, K, cus=256):  # noqa: F811
    stub.stub_form.argtypes = [ct.c_int64, ct.c_int, ct.c_int, ct.c_int64] + [ct.c_void_p] * 4
    v = [ct.c_int() for _ in range(4)]
    stub.stub_form(M, N, K, cus, *(ct.byref(x) for x in v))
    bm, mt, tn, parts = (x.value for x in v)
    return bm, (mt, tn), parts


@pytest.mark.parametrize("pieces,M,N,K", FEW)
def test_few_rows(stub, pieces, M, N, K):  # noqa: F811
    assert form(stub, M, N, K) == (0, pieces, 1)
    waves = WAVES[pieces][-1 if K > 4096 else 0]
    assert K // 128 > 2 * waves and K // 128 % waves != 0


def test_every_piece_is_listed():
    for pieces in WAVES:
        assert {K % 128 != 0 for p, _, _, K in FEW if p == pieces} == {False, True}


@pytest.mark.parametrize("bm,M,N,K", TILES + [(256, *s) for s in LARGE + STAY])
def test_tiles(stub, bm, M, N, K):  # noqa: F811
    assert form(stub, M, N, K) == (bm, (0, 0), 1)
    assert K >= 512


def test_who_stays():
    # whole pairs of steps and outputs of whole 16-byte pieces, in the shortest type
    for _, N, K in STAY:
        assert K % 256 == 0 and N * 2 % 16 == 0
    for _, N, K in LARGE:
        assert K % 256 != 0 or N * 4 % 16 != 0
    assert sum(-(-M // 256) * -(-N // 256) > 256 for M, N, _ in STAY) == 2


@pytest.mark.parametrize("parts,M,N,K", PARTS)
def test_parts(stub, parts, M, N, K):  # noqa: F811
    assert form(stub, M, N, K) == (128, (0, 0), parts)

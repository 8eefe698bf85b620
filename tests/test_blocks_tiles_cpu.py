"""That the sizes of test_blocks_tiles_gpu.py reach every kind of tiles, and what the query
that says so refuses. No GPU is needed.
"""
import ctypes
import os

import pytest

from linear_recurrent_sequence_amd import mlstm
from test_blocks_tiles_gpu import BF, FP, PRODUCTS, SIZES, tiles_of

pytestmark = pytest.mark.skipif(not os.path.exists(mlstm.LIB_PATH),
                                reason="libmlstm.so not built (run __graft_entry__.build())")

LARGE, MEDIUM, SMALL = (256, 256), (128, 256), (128, 128)
WHOLE, SPLIT, BOTH = "whole", "split", "both"
# (tile, form, whether a workgroup has several); what no size up to 16384 rows and widths of
# 8200 is taken in is left out
ALL = {(t, form, False) for t in (LARGE, MEDIUM, SMALL) for form in (WHOLE, SPLIT)} | {
    (t, form, True) for t in (LARGE, MEDIUM) for form in (WHOLE, SPLIT, BOTH)}
KINDS = {
    (BF, "forward"): ALL - {(LARGE, SPLIT, True)},
    (BF, "again"): ALL - {(LARGE, SPLIT, True)},
    (BF, "dx"): (ALL | {(SMALL, SPLIT, True)}) - {(SMALL, WHOLE, False)},
    (BF, "weights"): ALL | {(SMALL, WHOLE, True), (SMALL, SPLIT, True)},
    (FP, "forward"): ALL | {(SMALL, SPLIT, True)},
    (FP, "again"): ALL | {(SMALL, SPLIT, True)},
    (FP, "dx"): (ALL | {(SMALL, SPLIT, True)}) - {(SMALL, WHOLE, False)},
    (FP, "weights"): ALL | {(SMALL, WHOLE, True), (SMALL, SPLIT, True)},
}


def kind_of(size, dtype, product):
    tile, whole, split, shares = tiles_of(*size, dtype, product)
    form = WHOLE if split == 0 else SPLIT if whole == 0 else BOTH
    return tile, form, whole + split * shares > (512 if tile == SMALL else 256)


@pytest.mark.parametrize("dtype,product", KINDS)
def test_sizes_reach_every_kind_of_tiles(dtype, product):
    assert {kind_of(s, dtype, product) for s in SIZES[dtype]} >= KINDS[dtype, product]


@pytest.mark.parametrize("dtype", [BF, FP])
def test_tiles_cover_the_outputs_and_shares_the_workspace(dtype):
    bytes_of = mlstm.load_library().mlstm_gated_ffn_workspace_bytes
    for M, D, F in SIZES[dtype]:
        for product, p, q, groups in zip(PRODUCTS, (2 * F, 2 * F, D, D), (M, M, M, F), (1, 1, 1, 2)):
            (c, r), whole, split, shares = tiles_of(M, D, F, dtype, product)
            assert whole + split == -(-p // c) * -(-q // r) * groups
            assert shares == 1 if split == 0 else 2 <= shares <= 16
        if dtype == BF:  # the forward's only workspace
            (c, r), _, split, shares = tiles_of(M, D, F, dtype, "forward")
            assert bytes_of(M, D, F, mlstm.MLSTM_BF16, 0) == 4 * split * shares * c * r


def test_few_rows_have_no_tiles_and_what_is_refused():
    f = mlstm.load_library().mlstm_gated_ffn_tiles
    t = (ctypes.c_int64 * 5)(*[7] * 5)
    assert f(64, 64, 64, 1, 0, t) == 0 and list(t) == [0] * 5
    assert f(64, 64, 64, 1, 1, t) == 0 and t[0] > 0
    for args, status in (((0, 64, 64, 1, 0, t), -2), ((64, 60, 64, 1, 0, t), -4),
                         ((64, 64, 64, 2, 0, t), -3), ((64, 64, 64, 1, 4, t), -2),
                         ((64, 64, 64, 1, -1, t), -2), ((64, 64, 64, 1, 0, None), -1)):
        assert f(*args) == status

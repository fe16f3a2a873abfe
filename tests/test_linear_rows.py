"""The linear layer's kernel for few rows: the shapes that the GPU tests run reach every form of it, by rows of x and weight
tiles of a workgroup."""
import ctypes

import pytest

from block_quantized_matrix_amd import bqm
from tests.test_linear_tiles import TYPE, by_rows

I, I64 = ctypes.c_int, ctypes.c_int64
ROWS = (1, 4, 5, 16)
WIDTHS = (1999, 4201, 8301, 12403, 17501, 20507, 34901)  # one to eighteen eights of weight rows a workgroup, the last run short
# offsets, widths: runs of one row, and of up to sixteen; odd widths, so that matrices begin inside a tile of sixteen
GROUPS = [([0, 1, 1, 2, 3, 3], (601, 1451, 3203, 5003, 8003)), ([0, 1, 2, 3, 4, 5, 6, 7, 8], (401, 1531)),
          ([1, 10, 16], (601, 1451, 3203, 5003, 8003)), ([0, 5, 5, 16], (701, 2003))]


def kernel(x_type, grouped, R, N, groups=1):
    """(rows of x, weight tiles) of the workgroups of a call."""
    f = bqm.lib().bqm_internal_linear_rows_kernel
    f.argtypes, f.restype = [I, I, I64, I64, I64], I
    return divmod(f(TYPE[x_type], int(grouped), R, N, groups), 16)


@pytest.mark.parametrize("x_type", list(TYPE))
def test_every_kernel_has_a_shape(x_type):
    """One matrix and groups reach all of them, each for itself; 64 rows are covered by calls of 17 to 64 rows."""
    few = {(rm, t) for rm in (4, 16) for t in (1, 2, 3, 5, 9)}
    dense = {kernel(x_type, False, M, N) for M in ROWS for N in WIDTHS}
    grouped = {kernel(x_type, True, off[-1], N, min(len(off) - 1, off[-1])) for off, widths in GROUPS for N in widths}
    assert all(by_rows(x_type, False, M, N) for M in ROWS for N in WIDTHS)
    assert dense == few
    assert grouped == few
    for M, N in ((40, 150), (33, 1000), (64, 96)):
        assert by_rows(x_type, False, M, N) and kernel(x_type, False, M, N)[0] == (16 if x_type == "f32" else 64)

"""The linear layer's kernel and tile choices: the shapes that the GPU tests run reach every kernel and every tile."""
import ctypes

import pytest

from block_quantized_matrix_amd import bqm

Q4_0, Q8_0, MXFP4 = 2, 8, 39
F32, F16, BF16 = 0, 1, 30
FMT = {"q4_0": Q4_0, "q8_0": Q8_0, "mxfp4": MXFP4}
TYPE = {"f32": F32, "f16": F16, "bf16": BF16}
TILES = {"f32": 2, "f16": 5, "bf16": 5}
I, I64 = ctypes.c_int, ctypes.c_int64


def by_rows(x_type, grouped, R, N, groups=1):
    f = bqm.lib().bqm_internal_linear_rows
    f.argtypes, f.restype = [I, I, I64, I64, I64], I
    return bool(f(TYPE[x_type], int(grouped), R, N, groups))


def choice(fmt, x_type, grouped, R, N, K, groups=1):
    f = bqm.lib().bqm_internal_linear_choice
    f.argtypes, f.restype = [I, I, I, I64, I64, I64, I64], I
    return f(FMT[fmt], TYPE[x_type], int(grouped), R, N, K, groups)


def shapes(fmt, x_type):
    """For every tile a small (M, N) that takes it: N wide enough for its round of workgroups, K = 96 and 160 to be run."""
    found = {}
    for N in (4099, 8195, 16387, 33000):
        for M in (33, 70, 100, 130, 200, 300, 400, 600, 900):
            if not by_rows(x_type, False, M, N):
                c = choice(fmt, x_type, False, M, N, 4096)
                if c not in found and M * N <= 6_000_000:
                    found[c] = (M, N)
    return found


def grouped_shapes(fmt, x_type):
    """For every tile the mean rows of a group, over 40 groups of 1030 columns, that takes it."""
    found = {}
    for mean in (1, 3, 8, 14, 20, 30, 60):
        R, N, E = mean * 40, 1030, 40
        if not by_rows(x_type, True, R, N, E):
            found.setdefault(choice(fmt, x_type, True, R, N, 160, E), mean)
    return found


@pytest.mark.parametrize("x_type", list(TYPE))
@pytest.mark.parametrize("fmt", list(FMT))
def test_every_tile_has_a_shape(fmt, x_type):
    """Of one matrix and of groups together, as tests/test_gpu_linear_tiles.py runs them."""
    assert set(shapes(fmt, x_type)) | set(grouped_shapes(fmt, x_type)) == set(range(TILES[x_type]))


def test_few_rows_go_by_rows():
    assert by_rows("bf16", False, 16, 1 << 20) and not by_rows("bf16", False, 17, 8193)
    assert by_rows("bf16", False, 512, 1024) and not by_rows("bf16", False, 513, 1024)
    assert by_rows("f32", False, 64, 4096) and not by_rows("f32", False, 300, 4096)
    assert by_rows("bf16", True, 16, 4096, 128) and not by_rows("bf16", True, 17, 4096, 16)

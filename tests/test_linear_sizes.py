"""How large a call of the linear layer may be, as include/bqm.h states it: what it promises to take fits a launch, and what
does not fit is refused."""
import ctypes
import random

import pytest

from block_quantized_matrix_amd import bqm
from tests.test_linear import GROUPED, LINEAR, SHAPE, status
from tests.test_linear_tiles import FMT, TYPE

I, I64 = ctypes.c_int, ctypes.c_int64
MOST = (1 << 22) - 1  # workgroups of a launch


def workgroups(fmt, x_type, grouped, R, N, K, E=1):
    f = bqm.lib().bqm_internal_linear_workgroups
    f.argtypes, f.restype = [I, I, I, I64, I64, I64, I64], I64
    return f(FMT[fmt], TYPE[x_type], int(grouped), R, N, K, min(E, R) if grouped else 1)


def spread(rng, most):
    return int(2 ** rng.uniform(0, most))


@pytest.mark.parametrize("x_type", list(TYPE))
@pytest.mark.parametrize("fmt", list(FMT))
def test_sizes_that_are_promised_fit(fmt, x_type):
    rng = random.Random(f"{fmt} {x_type}")
    near = 0
    for _ in range(4000):
        K = 32 * spread(rng, 10)
        M = spread(rng, 24)
        N = min(1 << 30, max(1, int((1 << 22) / -(-M // 32) * 128 * rng.uniform(0.5, 1.0))))
        if -(-M // 32) * -(-N // 128) < 1 << 22:
            near += 1
            assert workgroups(fmt, x_type, False, M, N, K) <= MOST, (M, N, K)
        E, R = spread(rng, 12), spread(rng, 22)
        tiles = min(E + R // 32, R) + 16
        N = min((1 << 30) // E, max(1, int((1 << 22) / tiles * 128 * rng.uniform(0.5, 1.0))))
        if tiles * -(-N // 128) < 1 << 22:
            near += 1
            assert workgroups(fmt, x_type, True, R, N, K, E) <= MOST, (E, R, N, K)
    assert near > 4000


@pytest.mark.parametrize("name,base,sizes", [
    ("bqm_linear", LINEAR, dict(M=1, N=1 << 30, y_stride=1 << 30)),
    ("bqm_linear", LINEAR, dict(M=1 << 25, N=1 << 14, y_stride=1 << 14)),
    ("bqm_linear", LINEAR, dict(M=1 << 30, N=1024, y_stride=1024)),
    ("bqm_linear_grouped", GROUPED, dict(E=4096, R=4096, N=1 << 18, y_stride=1 << 18)),
    ("bqm_linear_grouped", GROUPED, dict(E=1, R=1 << 28, N=1 << 12, y_stride=1 << 12))])
def test_larger_calls_are_refused(name, base, sizes):
    """Where a launch does not hold the workgroups; none of these is promised."""
    c = dict(base, **sizes)
    grouped = name == "bqm_linear_grouped"
    rows, tiles = (c["R"], min(c["E"] + c["R"] // 32, c["R"]) + 16) if grouped else (c["M"], -(-c["M"] // 32))
    assert tiles * -(-c["N"] // 128) >= 1 << 22
    assert workgroups("q4_0", "f32", grouped, rows, c["N"], c["K"], c.get("E", 1)) > MOST
    assert status(name, base, **sizes) == SHAPE

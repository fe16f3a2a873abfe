"""The linear layer's kernel for few rows on the GPU: every form of it, exact on small integers, for one matrix and for
groups."""
import numpy as np
import pytest
import torch

from tests import _linref
from tests._gpu import DEV, say
from tests._linref import FMTS, TYPES
from tests.test_gpu_linear import f64, pack, run_grouped, run_linear
from tests.test_gpu_linear_tiles import integers
from tests.test_linear_rows import GROUPS, ROWS, WIDTHS

pytestmark = pytest.mark.gpu
BASE = 997  # different rows of weights; a prime, so that a row of another tile, run or matrix shows


def weights(fmt, N, K):
    """Packed weights of N rows, and their first BASE rows in fp64, which the others repeat."""
    b = integers(fmt, BASE, K, ("rows", K))
    return pack(fmt, np.ascontiguousarray(np.tile(b, (N // BASE + 1, 1, 1))[:N])), torch.from_numpy(_linref.dequantize(fmt, b)).to(DEV)


def whole(M, K, x_type):
    return torch.randint(-8, 9, (M, K), device=DEV).to(TYPES[x_type])


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [96, 160, 1056, 2208])
def test_every_kernel_is_exact_on_integers(K, fmt, x_type):
    """Sums of at most 2208 products below 2^7, in quarters: fp32 holds them all."""
    for N in WIDTHS:
        wp, W = weights(fmt, N, K)
        row = torch.arange(N, device=DEV) % BASE
        for M in ROWS:
            say("few rows", fmt, x_type, M, N, K)
            x = whole(M, K, x_type)
            room = torch.full((M + 1, N + 3), 7.0, device=DEV)
            y = room[:M, :N]
            run_linear(fmt, wp, x, y, M, N, K)
            assert torch.equal(y.double(), (x.double() @ W.t())[:, row])
            assert (room[:M, N:] == 7.0).all() and (room[M:] == 7.0).all()


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [96, 1056])
def test_every_kernel_in_groups(K, fmt, x_type):
    for off, widths in GROUPS:
        E, R = len(off) - 1, off[-1]
        cut = torch.tensor(off, dtype=torch.int32, device=DEV)
        for N in widths:
            say("few rows in groups", fmt, x_type, off, N, K)
            wp, W = weights(fmt, E * N, K)
            x = whole(R, K, x_type)
            y = torch.full((R, N), 7.0, device=DEV)
            run_grouped(fmt, wp, E, cut, x, y, R, N, K)
            want = torch.full((R, N), 7.0, dtype=torch.float64, device=DEV)
            for e in range(E):
                i, j = off[e], off[e + 1]
                want[i:j] = (x[i:j].double() @ W.t())[:, (torch.arange(N, device=DEV) + e * N) % BASE]
            assert torch.equal(y.double(), want)

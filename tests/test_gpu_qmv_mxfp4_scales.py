"""The MXFP4 decode product with scales at the end of their range: weights past fp32's largest number (scale bytes 253 and
254) count as what they are."""
import numpy as np
import pytest
import torch

import gen
from block_quantized_matrix_amd import bqm
from tests import _mxref
from tests._gpu import DEV, host, say
from tests.test_gpu_mxfp4 import blocks, close, packed

pytestmark = pytest.mark.gpu

# rows that give a compute unit one, two (half tiles and whole), three and more runs of eight
ROWS = [(48, 256), (4100, 160), (5125, 96), (8200, 64), (20011, 32), (34001, 32)]


def qmv(b, X):
    (N, nb), M = b.shape[:2], X.shape[0]
    Y = torch.full((M, N), 7.0, device=DEV)
    bqm.qmv_mxfp4(packed(b), torch.from_numpy(X).to(DEV), Y, M, N, nb * 32)
    return host(Y)


def product(b, X):
    return _mxref.product(_mxref.dequantize(b), X.astype(np.float64))


@pytest.mark.parametrize("M", [1, 5, 8])
@pytest.mark.parametrize("N,K", ROWS)
@pytest.mark.parametrize("lo,hi", [(253, 254), (240, 254), (80, 254)])
def test_largest_scales_with_small_inputs(M, N, K, lo, hi):
    """Sums far inside the range: inputs of one, two and three bf16 parts, and blocks of every scale in one row."""
    say("qmv largest scales", M, N, K, lo, hi)
    b = blocks(N, K, ("mxbig", N, lo), lo, hi)
    X = gen.normal((M, K), ("mxbig-x", M, K)).numpy()
    for x in (X, X.astype(np.float32).view(np.uint32) & np.uint32(0xFFFF0000), np.sign(X), np.zeros_like(X)):
        x = x.view(np.float32) if x.dtype == np.uint32 else x
        x = (x * np.float32(2.0 ** -40)).astype(np.float32)
        close(qmv(b, x), *product(b, x), K, "largest scales")


def test_one_weight_a_row():
    """Each code under each of the largest scales times inputs around 1: exact, infinite where fp32 ends."""
    say("qmv one weight a row")
    b = np.zeros((48, 5, 17), np.uint8)
    b[..., 0] = np.random.default_rng(1).integers(0, 253, (48, 5))  # of zero codes
    for r in range(48):
        at = 7 * r % 160
        b[r, at // 32, 0] = 252 + r // 16
        b[r, at // 32, 1 + at % 16] = r % 16 << (4 if at % 32 >= 16 else 0)
    W = _mxref.dequantize(b)
    for x in (1.0, 0.25, -0.5, 0.125 + 2.0 ** -12 + 2.0 ** -20, 2.0 ** -130, -1.5, 3.0e-30):
        X = np.full((2, 160), x, np.float32)
        with np.errstate(over="ignore"):
            want = (X.astype(np.float64) @ W.T).astype(np.float32)
        assert np.array_equal(qmv(b, X), want), x


def test_smallest_scales_beside_them():
    """Blocks of the largest scales whose codes are 0 take nothing from blocks of the smallest in the same row."""
    say("qmv smallest beside largest scales")
    b = blocks(40, 256, ("mxbig-z",), 0, 3)
    b[:, ::3, 0], b[:, ::3, 1:] = 254, 0
    X = (gen.normal((3, 256), ("mxbig-zx",)).numpy() * 2.0 ** 60).astype(np.float32)
    close(qmv(b, X), *product(b, X), 256, "smallest beside largest")


@pytest.mark.parametrize("M", [1, 8])
def test_special_values_beside_them(M):
    say("qmv largest scales, specials", M)
    b = blocks(33, 192, ("mxbig-s",), 253, 254)
    b[8:20, :, 0] = 120                       # rows of ordinary scales in the same tiles
    X = (gen.normal((M, 192), ("mxbig-sx", M)).numpy() * 2.0 ** -40).astype(np.float32)
    b[3, 1, 0] = b[9, 4, 0] = 255              # a NaN scale: its row and no other
    close(qmv(b, X), *product(b, X), 192, "NaN scales")
    b[3, 1, 0] = b[9, 4, 0] = 254
    for v in (np.inf, -np.inf, np.nan):       # an input: infinite by the sign of its weight, NaN where that is 0
        X[M - 1, 70] = v
        got, w = qmv(b, X), _mxref.dequantize(b)[:, 70]
        assert np.isfinite(got[:M - 1]).all()
        with np.errstate(invalid="ignore"):
            assert np.array_equal(got[M - 1], (w * v).astype(np.float32), equal_nan=True)

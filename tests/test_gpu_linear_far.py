"""Tiles beside numbers far from 1: MXFP4 scales so small that weights are subnormal in bf16, under rows that bring them back,
and rows so small that their parts are, under scales that do."""
import numpy as np
import pytest
import torch

from tests import _linref
from tests._gpu import DEV, say
from tests._linref import TYPES
from tests.test_gpu_linear import f64, pack, rows, run_linear

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x_type", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(70, 4099), (600, 4099)])
@pytest.mark.parametrize("lowest,size", [(0, 2.0 ** 100), (2, 2.0 ** 90), (240, 2.0 ** -125), (250, 2.0 ** -130)])
def test_far_scales_and_rows(lowest, size, M, N, x_type):
    """Rows of bf16 are made of its own numbers, subnormal ones among them; of fp32 rows what is below 2^-133 is left out."""
    say("far", lowest, size, M, N, x_type)
    K = 192
    b = _linref.blocks("mxfp4", N, K, ("far-t", lowest))
    b[..., 0] = lowest + np.arange(N * K // 32).reshape(N, -1) % 3
    W = _linref.dequantize("mxfp4", b)
    x = (rows(M, K, ("far-tx", M), torch.float32) * size).to(TYPES[x_type])
    y = torch.empty((M, N), device=DEV)
    run_linear("mxfp4", pack("mxfp4", b), x, y, M, N, K)
    Y, S = _linref.linear(W, f64(x))
    tol = _linref.tolerance(Y, S, K, torch.float32)
    if x_type == "f32":
        tol = tol + 2.0 ** -133 * np.abs(W).sum(1)
    _linref.close(f64(y), Y, tol, f"{lowest} {size} {x_type}")
    if size > 1:  # not drowned in the tolerance
        assert np.median(tol / np.abs(Y)) < 1e-2

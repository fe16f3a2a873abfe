"""The embedding's scale over all of fp32's range beside MXFP4's block scales over theirs: one rounding whatever the two are."""
import numpy as np
import pytest
import torch

from block_quantized_matrix_amd import bqm
from tests import _linref
from tests._gpu import DEV, host, say
from tests.test_gpu_linear import pack

pytestmark = pytest.mark.gpu
SCALES = [1.2e-40, 2.0 ** -149, 2.0 ** -126 * 1.7, -7e-39, 1.0 / 3, 2.0 ** 125 * 1.1, 3.4e38, -2.0 ** 127, 0.0]


@pytest.mark.parametrize("scale", SCALES)
def test_embed_scale(scale):
    """The product is rounded to 24 bits, and once more, to half of 2^-149, where it is below 2^-126."""
    say("embed scale", scale)
    b = np.zeros((256, 1, 17), np.uint8)
    b[:, 0, 0] = np.arange(256)
    b[:, 0, 1:] = np.arange(16) | np.arange(16)[::-1] << 4
    W, ids = _linref.dequantize("mxfp4", b), torch.arange(256, dtype=torch.int32, device=DEV)
    y = torch.empty((256, 32), device=DEV)
    bqm.bqm_embed("mxfp4", pack("mxfp4", b), 256, 32, ids, 256, scale, y, 32)
    want, got = W * np.float64(np.float32(scale)), host(y).astype(np.float64)
    top = 2.0 ** 128 * (1 - 2.0 ** -25)  # from here on the nearest number of fp32 is an infinity
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inside = np.abs(want) < top
    assert np.array_equal(got[np.abs(want) >= top], np.sign(want[np.abs(want) >= top]) * np.inf)
    assert (np.abs(got - want)[inside] <= np.abs(want)[inside] * 2.0 ** -24 + 2.0 ** -150).all()


def test_embed_scale_not_finite():
    """As the formula: every number of the table times an infinity or NaN."""
    say("embed scale not finite")
    b = _linref.blocks("mxfp4", 8, 64, ("nf",))
    W, ids = _linref.dequantize("mxfp4", b), torch.arange(8, dtype=torch.int32, device=DEV)
    for scale in (float("inf"), -float("inf"), float("nan")):
        y = torch.empty((8, 64), device=DEV)
        bqm.bqm_embed("mxfp4", pack("mxfp4", b), 8, 64, ids, 8, scale, y, 64)
        with np.errstate(invalid="ignore"):
            assert np.array_equal(host(y), (W * scale).astype(np.float32), equal_nan=True)

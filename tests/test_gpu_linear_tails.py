"""The activations far below 0, where they are smaller than fp32's step at 1 but not 0: a large mul brings them up."""
import numpy as np
import pytest
import torch

from block_quantized_matrix_amd import bqm
from tests import _linref
from tests._gpu import DEV, host, say

pytestmark = pytest.mark.gpu
LOWEST = {"silu": -110.0, "gelu": -15.0, "gelu_tanh": -11.5}  # below these nothing is left of a number of fp32


@pytest.mark.parametrize("M", [1, 40, 300])  # rows by rows, by tiles of whole fours and of columns that are none
@pytest.mark.parametrize("N", [4099, 4100])
@pytest.mark.parametrize("act", list(LOWEST))
def test_tails_are_kept(act, M, N):
    """With K = 0 z is the bias itself.  The value's error: its exponent t (of silu z, of the tanh form 1.6 (|z| +
    0.0447 |z|^3), of erfc z^2 / 2 with twice its relative error) is rounded six times at most, counting |t| 2^-24
    each, or z^2 2^-24 twice; exponential, reciprocal and products take eight half steps more.  A number below 2^-126 is
    rounded to a multiple of 2^-149, erfc itself before it is multiplied by |z| / 2.  Then the product with mul."""
    say("tails", act, M, N)
    low = LOWEST[act]
    z = torch.cat([torch.linspace(low, low / 4, N - 40), torch.linspace(-1e30, 5.0, 40)]).float().to(DEV)
    mul = torch.full((M, N), 2.0 ** 100, device=DEV)
    y = torch.empty((M, N), device=DEV)
    bqm.bqm_linear("q8_0", None, torch.empty((M, 0), device=DEV), 0, y, N, M, N, 0, bias=z, act=act, mul=mul, mul_stride=N)
    z = host(z).astype(np.float64)
    want = _linref.act(act, z)
    t = {"silu": np.abs(z), "gelu": z * z / 2, "gelu_tanh": 1.6 * (np.abs(z) + 0.0447 * np.abs(z) ** 3)}[act]
    with np.errstate(over="ignore"):
        tol = (np.minimum(6 * t, 2000) + 8) * 2.0 ** -24 * np.abs(want) + 2.0 ** -150 * (1 + np.minimum(np.abs(z), 20) / 2)
    got = host(y).astype(np.float64) / 2.0 ** 100
    assert (got == got[:1]).all()
    bad = ~(np.abs(got[0] - want) <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {N}, z = {z[bad][:3]}: {got[0][bad][:3]}, not {want[bad][:3]}"

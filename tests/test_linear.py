"""bqm_embed, bqm_linear and bqm_linear_grouped on the host: what they refuse, before anything is launched."""
import ctypes
import types

import numpy as np
import pytest
import torch

from block_quantized_matrix_amd import bqm
from tests import _linref

P = ctypes.c_void_p
GOOD, ODD, ODD4 = P(0x100000), P(0x100008), P(0x100002)  # never dereferenced on these paths
OK, NULL, SHAPE, ALIGN, UNSUPPORTED = 0, 1, 2, 3, 4

EMBED = dict(fmt=2, w=GOOD, rows=10, K=64, ids=GOOD, T=3, scale=1.0, y_type=0, Y=GOOD, y_stride=64)
LINEAR = dict(fmt=2, w=GOOD, x_type=0, X=GOOD, x_stride=64, bias=None, act=0, mul=None, mul_stride=0, res=None, res_stride=0,
              y_type=0, Y=GOOD, y_stride=8, M=3, N=8, K=64)
GROUPED = dict(fmt=2, w=GOOD, E=4, offsets=GOOD, x_type=0, X=GOOD, x_stride=64, bias=None, act=0, mul=None, mul_stride=0,
               res=None, res_stride=0, y_type=0, Y=GOOD, y_stride=8, R=3, N=8, K=64)


def status(name, base, **change):
    assert set(change) <= set(base)
    return getattr(bqm.lib(), name)(*dict(base, **change).values(), None)


@pytest.mark.parametrize("change,want", [
    (dict(fmt=3), UNSUPPORTED), (dict(y_type=2), UNSUPPORTED), (dict(y_type=-1), UNSUPPORTED),
    (dict(rows=-1), SHAPE), (dict(rows=(1 << 30) + 1), SHAPE), (dict(K=40), SHAPE), (dict(K=-32), SHAPE), (dict(T=-1), SHAPE),
    (dict(T=(1 << 30) + 1), SHAPE), (dict(y_stride=63), SHAPE), (dict(y_stride=(1 << 30) + 1), SHAPE),
    (dict(ids=None), NULL), (dict(Y=None), NULL), (dict(w=None), NULL), (dict(ids=ODD), ALIGN), (dict(Y=ODD), ALIGN),
    (dict(w=ODD), ALIGN), (dict(T=0, ids=None, Y=None), OK), (dict(K=0, ids=None, Y=None), OK)])
def test_embed_refuses(change, want):
    assert status("bqm_embed", EMBED, **change) == want


COMMON = [
    (dict(fmt=3), UNSUPPORTED), (dict(x_type=2), UNSUPPORTED), (dict(y_type=7), UNSUPPORTED), (dict(act=5), UNSUPPORTED),
    (dict(act=-1), UNSUPPORTED), (dict(N=-1), SHAPE), (dict(N=(1 << 30) + 1, y_stride=1 << 30), SHAPE), (dict(K=48), SHAPE),
    (dict(K=-32), SHAPE), (dict(K=(1 << 20) + 32, x_stride=(1 << 20) + 32), SHAPE), (dict(x_stride=32), SHAPE),
    (dict(x_stride=(1 << 20) + 8), SHAPE), (dict(y_stride=7), SHAPE), (dict(y_stride=(1 << 30) + 1), SHAPE),
    (dict(mul=GOOD, mul_stride=7), SHAPE), (dict(res=GOOD, res_stride=7), SHAPE),
    (dict(mul=GOOD, mul_stride=(1 << 30) + 1), SHAPE), (dict(res=GOOD, res_stride=(1 << 30) + 1), SHAPE),
    (dict(w=None), NULL), (dict(X=None), NULL), (dict(Y=None), NULL), (dict(w=ODD), ALIGN), (dict(X=ODD), ALIGN),
    (dict(Y=ODD), ALIGN), (dict(mul=ODD, mul_stride=8), ALIGN), (dict(res=ODD, res_stride=8), ALIGN), (dict(bias=ODD4), ALIGN),
    (dict(x_stride=66), ALIGN), (dict(x_type=1, x_stride=68), ALIGN), (dict(N=0, Y=None, y_stride=0), OK),
    (dict(N=1 << 30, y_stride=1 << 30), SHAPE)]  # more workgroups than a launch holds


@pytest.mark.parametrize("change,want", COMMON + [(dict(M=-1), SHAPE), (dict(M=(1 << 30) + 1), SHAPE), (dict(M=0, X=None, Y=None), OK)])
def test_linear_refuses(change, want):
    assert status("bqm_linear", LINEAR, **change) == want


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(E=-1), SHAPE), (dict(E=4097), SHAPE), (dict(E=4096, N=1 << 19, y_stride=1 << 19), SHAPE), (dict(offsets=None), NULL),
    (dict(offsets=ODD), ALIGN), (dict(R=-1), SHAPE), (dict(R=(1 << 30) + 1), SHAPE), (dict(R=0, X=None, Y=None), OK),
    (dict(E=0, offsets=None, Y=None), OK)])
def test_grouped_refuses(change, want):
    assert status("bqm_linear_grouped", GROUPED, **change) == want


def test_binding_refuses_types():
    """An operand of another type than it has to be is refused, whatever its shape."""
    w = torch.zeros(4096, dtype=torch.uint8)
    f32, f16, i64 = torch.zeros(2, 64), torch.zeros(2, 64, dtype=torch.float16), torch.zeros(64, dtype=torch.int64)

    def refused(call, *args, **more):
        with pytest.raises(bqm.BqmError) as e:
            call(*args, stream=types.SimpleNamespace(cuda_stream=None), **more)
        assert e.value.status == UNSUPPORTED

    linear = lambda **more: bqm.bqm_linear("q4_0", w, f32, 64, f32, 64, 2, 64, 64, **more)  # noqa: E731
    refused(linear, bias=f16)
    refused(linear, mul=f16, mul_stride=64)
    refused(linear, residual=f16, res_stride=64)
    refused(linear, act="tanh")
    refused(bqm.bqm_linear, "q4_0", w, i64, 64, f32, 64, 2, 64, 64)
    refused(bqm.bqm_linear_grouped, "q4_0", w, 1, i64, f32, 64, f32, 64, 2, 64, 64)
    refused(bqm.bqm_embed, "q4_0", w, 4, 64, i64, 2, 1.0, f32, 64)


@pytest.mark.parametrize("fmt", _linref.FMTS)
def test_reference_decodes_by_the_definition(fmt):
    """The plain form's weights, value by value from the bytes."""
    b = _linref.blocks(fmt, 3, 64, ("ref",))
    W = _linref.dequantize(fmt, b)
    grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for r in range(3):
        for k in range(64):
            blk, j = b[r, k // 32], k % 32
            if fmt == "q8_0":
                want = float(np.int8(blk[2 + j])) * float(blk[:2].view(np.float16)[0])
            else:
                c = int(blk[-16 + j % 16]) >> (4 * (j // 16)) & 15
                want = (c - 8) * float(blk[:2].view(np.float16)[0]) if fmt == "q4_0" else \
                    (-1) ** (c >> 3) * grid[c & 7] * 2.0 ** (int(blk[0]) - 127)
            assert W[r, k] == want

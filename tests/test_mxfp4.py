"""The MXFP4 calls and the router on the host: sizes, refusals before any launch, and the plain forms that the GPU tests
compare with, against hand-worked values.  No GPU needed."""
import ctypes
import types

import numpy as np
import pytest

from block_quantized_matrix_amd import bqm
from tests import _mxref

P = ctypes.c_void_p
GOOD = P(0x100000)  # aligned stand-ins, never dereferenced: every call below ends before a launch
ODD = P(0x100008)
NULL, SHAPE, ALIGN, UNSUPPORTED = 1, 2, 3, 4
F32, F16, BF16 = 0, 1, 30


def test_packed_bytes():
    # 16-row tiles: 1024 code bytes per 128 of K, 256 scale bytes per 512 of K
    assert bqm.packed_bytes("mxfp4", 1, 32) == 1024 + 256
    assert bqm.packed_bytes("mxfp4", 16, 128) == 1024 + 256
    assert bqm.packed_bytes("mxfp4", 17, 544) == 2 * (5 * 1024 + 2 * 256)
    assert bqm.packed_bytes("mxfp4", 4096, 4096) == 4096 * 4096 * 17 // 32
    assert bqm.packed_bytes("mxfp4", 0, 64) == bqm.packed_bytes("mxfp4", 4, 0) == 0
    assert bqm.packed_bytes("mxfp4", 4, 48) == bqm.packed_bytes("mxfp4", -1, 64) == 0


def test_other_products_refuse_the_format():
    L, f = bqm.lib(), bqm.MXFP4
    assert L.qmv_id(f, GOOD, 4, 8, 64, GOOD, 1, 2, GOOD, 64, 0, GOOD, None) == UNSUPPORTED
    assert L.qmv_id_gate_up(f, GOOD, GOOD, 4, 8, 64, GOOD, 1, 2, GOOD, 64, 0, GOOD, None) == UNSUPPORTED
    assert L.qmv_id_sum(f, GOOD, 4, 8, 64, GOOD, GOOD, 1, 2, GOOD, 64, 0, GOOD, GOOD, None) == UNSUPPORTED
    assert L.qmv_id_sum_noalloc(f, GOOD, 4, 8, 64, GOOD, GOOD, 1, 2, GOOD, 64, 0, GOOD, None) == UNSUPPORTED
    assert L.qmm_id(f, GOOD, 4, 8, 64, GOOD, 1, 2, GOOD, GOOD, 1, 0, GOOD, None) == UNSUPPORTED
    assert L.qmv_chain(f, 1, GOOD, 1, None) == UNSUPPORTED
    arr = (bqm.Gemv * 1)(bqm.Gemv(0x10000, 0x10000, 0x10000, 64, 64, f, 0, 1, 0))
    assert L.bqm_chain_prepare(ctypes.cast(arr, P), 1, P(0x20000), None) == UNSUPPORTED


def test_repack_refusals():
    L, f = bqm.lib(), bqm.MXFP4
    for call in (lambda a, b, r, k: L.bqm_repack(f, a, b, r, k, None), lambda a, b, r, k: L.bqm_unpack(f, b, a, r, k, None)):
        assert call(GOOD, GOOD, 4, 48) == SHAPE
        assert call(GOOD, GOOD, -1, 64) == SHAPE
        assert call(None, GOOD, 4, 64) == NULL
        assert call(GOOD, None, 4, 64) == NULL
        assert call(GOOD, ODD, 4, 64) == ALIGN
        assert call(None, None, 0, 64) == 0


def test_quantize_refusals():
    L = bqm.lib()
    for call in (lambda t, x, st, p, r, k: L.bqm_quantize_mxfp4(t, x, st, p, r, k, None),
                 lambda t, x, st, p, r, k: L.bqm_dequantize_mxfp4(p, t, x, st, r, k, None)):
        assert call(7, GOOD, 64, GOOD, 4, 64) == UNSUPPORTED
        assert call(-1, GOOD, 64, GOOD, 4, 64) == UNSUPPORTED
        assert call(F32, GOOD, 48, GOOD, 4, 48) == SHAPE
        assert call(F32, GOOD, 63, GOOD, 4, 64) == SHAPE
        assert call(F32, GOOD, 64, GOOD, -4, 64) == SHAPE
        assert call(F32, GOOD, (1 << 30) + 1, GOOD, 4, 64) == SHAPE
        assert call(F16, None, 64, GOOD, 4, 64) == NULL
        assert call(BF16, GOOD, 64, None, 4, 64) == NULL
        assert call(F32, ODD, 64, GOOD, 4, 64) == ALIGN
        assert call(F32, GOOD, 64, ODD, 4, 64) == ALIGN
        assert call(F32, None, 64, None, 0, 64) == 0
        assert call(F32, None, 0, None, 4, 0) == 0


def test_product_refusals():
    L = bqm.lib()
    assert L.qmv_mxfp4(GOOD, GOOD, GOOD, 9, 64, 64, None) == SHAPE
    assert L.qmv_mxfp4(GOOD, GOOD, GOOD, -1, 64, 64, None) == SHAPE
    assert L.qmv_mxfp4(GOOD, GOOD, GOOD, 1, 64, 40, None) == SHAPE
    assert L.qmv_mxfp4(GOOD, GOOD, GOOD, 1, (1 << 30) + 1, 64, None) == SHAPE
    for f in (lambda w, x, y: L.qmv_mxfp4(w, x, y, 1, 64, 64, None), lambda w, x, y: L.qmm_mxfp4(w, x, y, 1, 64, 64, None),
              lambda w, x, y: L.qmm_id_mxfp4(w, 4, 64, 64, GOOD, 1, 2, x, 1, 1, 0, y, None)):
        for at in range(3):
            for bad, status in ((None, NULL), (ODD, ALIGN)):
                assert f(*[bad if i == at else GOOD for i in range(3)]) == status
    assert L.qmv_mxfp4(GOOD, GOOD, GOOD, 1, (1 << 29) + 1, 64, None) == SHAPE
    assert L.qmv_mxfp4(GOOD, GOOD, GOOD, 1, 64, (1 << 23) + 32, None) == SHAPE
    assert L.qmm_mxfp4(GOOD, GOOD, GOOD, 1, 64, (1 << 23) + 32, None) == SHAPE
    assert L.qmm_mxfp4(GOOD, GOOD, GOOD, 1 << 30, 64, 64, None) == SHAPE  # 2^22 tiles
    assert L.qmm_mxfp4(GOOD, GOOD, GOOD, -1, 64, 64, None) == SHAPE
    assert L.qmm_mxfp4(GOOD, GOOD, GOOD, 1, 64, 33, None) == SHAPE
    assert L.qmv_mxfp4(None, None, None, 0, 64, 64, None) == 0
    assert L.qmv_mxfp4(None, None, None, 1, 0, 64, None) == 0
    assert L.qmm_mxfp4(None, None, None, 0, 64, 64, None) == 0
    assert L.qmm_mxfp4(None, None, None, 64, 0, 64, None) == 0


def test_product_id_refusals():
    L = bqm.lib()

    def call(E=4, N=64, K=64, ids=GOOD, T=2, k=2, rows=4, xt=2, xs=1):
        return L.qmm_id_mxfp4(GOOD, E, N, K, ids, T, k, GOOD, rows, xt, xs, ODD, None)

    assert call() == ALIGN  # only Y is wrong
    assert call(rows=3) == SHAPE  # the last slot's row lies outside
    assert call(T=16385) == call(k=33) == call(E=4097) == call(N=-1) == call(K=48) == call(E=-1) == SHAPE
    assert call(xt=-1) == call(xs=-1) == call(xt=(1 << 30) + 1) == call(rows=-1) == SHAPE
    assert call(N=1 << 30) == SHAPE
    assert call(ids=ODD) == ALIGN
    assert L.qmm_id_mxfp4(GOOD, 4, 64, 64, None, 2, 2, GOOD, 4, 2, 1, GOOD, None) == NULL
    assert call(T=0, rows=0) == call(k=0, rows=0) == call(N=0) == 0


def test_route_refusals():
    L = bqm.lib()

    def call(score=0, t=F32, logits=GOOD, stride=64, bias=None, T=2, E=64, g=1, kg=1, gt=1, k=4, ids=GOOD, w=ODD):
        return L.bqm_route(score, t, logits, stride, bias, T, E, g, kg, gt, k, 1, 1.0, ids, w, None)

    assert call() == ALIGN  # only the weights are wrong
    assert call(score=2) == call(t=2) == UNSUPPORTED
    assert call(T=-1) == call(T=(1 << 22) + 1) == call(E=4097, stride=4097) == call(k=33) == call(k=-1) == SHAPE
    assert call(stride=63) == call(stride=(1 << 30) + 1) == SHAPE
    assert call(g=0) == call(g=3) == call(g=65, E=65, stride=65) == call(g=4, kg=0) == call(g=4, kg=5) == SHAPE
    assert call(gt=0) == call(gt=3) == call(g=64, kg=8, gt=2) == SHAPE
    assert call(logits=None, w=GOOD) == call(ids=None) == call(w=None) == NULL
    assert call(logits=ODD, w=GOOD) == call(ids=ODD) == call(bias=P(0x100002), w=GOOD) == ALIGN
    assert call(T=0) == call(k=0) == 0


def test_binding_refuses_other_types():
    import torch
    x = torch.zeros((1, 32), dtype=torch.float64)
    with pytest.raises(bqm.BqmError) as e:
        bqm.bqm_quantize_mxfp4(x, 32, x, 1, 32, stream=types.SimpleNamespace(cuda_stream=0))
    assert e.value.status == UNSUPPORTED


def test_reference_by_hand():
    x = np.zeros((1, 64))
    x[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]  # largest 6: scale 1; ties go to the even code
    x[0, 16] = -7.9                                       # beyond 6: kept at -6, scale still 1
    x[0, 32:34] = [2.0 ** -140, -2.0 ** -127]             # scale held at 2^-127
    b = _mxref.quantize(x)
    assert b.shape == (1, 2, 17)
    assert b[0, 0, 0] == 127 and list(b[0, 0, 1:9]) == [0x7 | 0xF0, 0, 2, 2, 4, 4, 6, 6]
    assert b[0, 1, 0] == 0 and list(b[0, 1, 1:3]) == [0, 0xA]
    back = _mxref.dequantize(b)
    assert list(back[0, :8]) == [6, 0, 1, 1, 2, 2, 4, 4] and back[0, 16] == -6 and back[0, 33] == -2.0 ** -127
    x[0, 40] = np.inf
    assert np.isnan(_mxref.dequantize(_mxref.quantize(x))[0, 32:]).all()


def test_route_reference_by_hand():
    inf = np.inf
    l = np.array([[1.0, 3, 3, -inf, 2, 0], [0, -inf, -inf, -inf, -inf, -inf], [np.nan, 0, 0, 0, 0, 0]])
    ids, w = _mxref.route(l, None, "softmax", 1, 1, 1, 3, True, 2.0)
    assert ids.tolist() == [[1, 2, 4], [0, -1, -1], [0, 1, 2]]
    z = np.exp([3, 3, 2])
    assert np.allclose(w[0], 2 * z / z.sum()) and w[1].tolist() == [2, 0, 0] and np.isnan(w[2]).all()
    # two groups of three, sums of the best two scores: group 0 holds 3 and 3
    ids, _ = _mxref.route(l[:1], None, "sigmoid", 2, 1, 2, 4, False, 1.0)
    assert ids.tolist() == [[1, 2, 0, -1]]


def test_text_of_unsupported():
    """The status that an unknown format, element type or score gets says so."""
    for word in ("format", "type", "score"):
        assert word in bqm.strerror(UNSUPPORTED)

"""Every tile of the MXFP4 products at sizes that it does not divide, against the products in 64 bits (made on the GPU)."""
import numpy as np
import pytest
import torch

import gen
from block_quantized_matrix_amd import bqm
from tests import _mxref, _tiles
from tests._gpu import DEV, host, say
from tests.test_gpu_mxfp4 import blocks, packed

pytestmark = pytest.mark.gpu


def dequantized(b):
    b = torch.from_numpy(b).to(DEV)
    table = torch.tensor(np.r_[_mxref.GRID, -_mxref.GRID], device=DEV)
    codes = torch.cat([b[..., 1:] & 15, b[..., 1:] >> 4], -1).to(torch.int32)
    scale = torch.from_numpy(np.ldexp(1.0, np.arange(256) - 127)).to(DEV)
    return (table[codes] * scale[b[..., :1].to(torch.int32)]).reshape(b.shape[0], -1)


def product(W, X):
    """Y = X W^T and the sum of the terms' magnitudes, 64 bits."""
    return X @ W.t(), X.abs() @ W.abs().t()


def close(Y, want, S, K, what):
    bad = ~((Y.double() - want).abs() <= _mxref.tolerance(K) * S)
    assert not bad.any(), f"{what}: {int(bad.sum())} outputs off, the first at {bad.nonzero()[:4].tolist()}"


def outputs(*shape):
    """Outputs with room behind them that has to stay as it is."""
    n = int(np.prod(shape))
    y = torch.full((n + 64,), 7.0, device=DEV)
    return y, y[:n].view(shape)


@pytest.mark.parametrize("tile,M,N,K", _tiles.DENSE)
def test_dense(tile, M, N, K):
    say("qmm_mxfp4 tile", tile, M, N, K)
    assert _tiles.dense_choice(M, N, K) == tile
    w, x = blocks(N, K, ("mxtile", N, K)), blocks(M, K, ("mxtile-x", M, K))
    room, Y = outputs(M, N)
    bqm.qmm_mxfp4(packed(w), packed(x), Y, M, N, K)
    close(Y, *product(dequantized(w), dequantized(x)), K, "qmm")
    assert (host(room[M * N:]) == 7.0).all()


@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("tile,T,E,top_k,N,K", _tiles.INDEXED)
def test_indexed(tile, T, E, top_k, N, K, per_slot):
    say("qmm_id_mxfp4 tile", tile, T, E, top_k, N, K, per_slot)
    assert _tiles.indexed_choice(E, N, T * top_k) == tile
    w = blocks(E * N, K, ("mxtile-i", E, N, K))
    ids = gen.router_ids(T, E, top_k, ("mxtile-ids", T, E))
    ids.reshape(-1)[3::11], ids.reshape(-1)[5::13] = -1, E + 2
    rows, (xt, xs) = (T * top_k, (top_k, 1)) if per_slot else (T, (1, 0))
    x = blocks(rows, K, ("mxtile-ix", rows, K))
    room, Y = outputs(T * top_k, N)
    bqm.qmm_id_mxfp4(packed(w), E, N, K, torch.from_numpy(ids).to(DEV), T, top_k, packed(x), rows, xt, xs, Y)
    W, X, flat = dequantized(w), dequantized(x), ids.reshape(-1)
    X = X if per_slot else X.repeat_interleave(top_k, 0)
    for e in range(E):
        mine = torch.from_numpy(np.flatnonzero(flat == e)).to(DEV)
        if len(mine):
            close(Y[mine], *product(W[e * N:(e + 1) * N], X[mine]), K, f"qmm_id, expert {e}")
    Y = host(Y)
    assert (Y[flat < 0] == 0).all() and np.isnan(Y[flat >= E]).all() and (host(room[T * top_k * N:]) == 7.0).all()


@pytest.mark.parametrize("M", [1, 5, 8])
@pytest.mark.parametrize("runs,N", list(_tiles.DECODE.items()))
def test_decode(runs, N, M):
    """K in eleven steps, which neither eight nor sixteen waves share evenly."""
    say("qmv_mxfp4 runs", runs, N, M)
    assert _tiles.decode_runs(N) == runs
    for K in (1312, 128 * 19):
        b = blocks(N, K, ("mxruns", N))
        X = gen.normal((M, K), ("mxruns-x", M, K), device=DEV)
        room, Y = outputs(M, N)
        bqm.qmv_mxfp4(packed(b), X, Y, M, N, K)
        close(Y, *product(dequantized(b), X.double()), K, "qmv")
        assert (host(room[M * N:]) == 7.0).all()


def test_largest_k():
    """Rows of the longest K that the products take, quantized, multiplied and given back."""
    K, N, M = 1 << 23, 17, 3
    say("largest K", K)
    g = torch.Generator(DEV).manual_seed(3)
    b = torch.randint(0, 256, (N + M, K // 32, 17), dtype=torch.uint8, device=DEV, generator=g)
    b[..., 0] = torch.randint(118, 133, (N + M, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    b = host(b)
    w, x, W, X = packed(b[:N]), packed(b[N:]), dequantized(b[:N]), dequantized(b[N:])
    Y = torch.empty((M, N), device=DEV)
    bqm.qmm_mxfp4(w, x, Y, M, N, K)
    close(Y, *product(W, X), K, "qmm")
    Y.zero_()
    bqm.qmv_mxfp4(w, X.float(), Y, M, N, K)
    close(Y, *product(W, X), K, "qmv")
    Y = torch.zeros((M, 1, N), device=DEV)
    bqm.qmm_id_mxfp4(w, 1, N, K, torch.zeros((M, 1), dtype=torch.int32, device=DEV), M, 1, x, M, 1, 0, Y)
    close(Y[:, 0], *product(W, X), K, "qmm_id")
    back, again = torch.empty((M, K), device=DEV), torch.zeros_like(x)
    bqm.bqm_dequantize_mxfp4(x, back, K, M, K)
    assert torch.equal(back.double(), X)
    bqm.bqm_quantize_mxfp4(back, K, again, M, K)
    bqm.bqm_dequantize_mxfp4(again, back, K, M, K)
    assert torch.equal(back.double(), torch.from_numpy(_mxref.dequantize(_mxref.quantize(host(X)))).to(DEV))

"""The linear layer's tiles on the GPU, every one of them for every format and type, exact on small integers and against
the plain 64-bit form; the short K at which a tile's pipeline starts and ends, odd numbers of blocks among them."""
import numpy as np
import pytest
import torch

import gen
from block_quantized_matrix_amd import bqm
from tests import _linref
from tests._gpu import DEV, say
from tests._linref import FMTS, TYPES
from tests.test_gpu_graphs import replays_match_eager
from tests.test_gpu_linear import check, f64, pack, rows, run_grouped, run_linear
from tests.test_linear_tiles import grouped_shapes, shapes

pytestmark = pytest.mark.gpu


def integers(fmt, N, K, key):
    """Blocks whose products with small integers leave nothing to round."""
    b = _linref.blocks(fmt, N, K, key)
    g = np.random.default_rng(gen.seed_of("tiles", *key))
    if fmt == "mxfp4":
        b[..., 0] = g.integers(126, 129, (N, K // 32))
    else:
        b[..., :2] = g.choice(np.array([0.5, 1, 2, -1], np.float16), (N, K // 32))[..., None].view(np.uint8)
        if fmt == "q8_0":
            b[..., 2:] = g.integers(-9, 10, (N, K // 32, 32)).astype(np.int8).view(np.uint8)
    return b


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("fmt", FMTS)
def test_every_tile_is_exact_on_integers(fmt, x_type):
    found = shapes(fmt, x_type)
    for c, (M, N) in sorted(found.items()):
        for K in (32, 96, 160, 320):
            say("tile", c, fmt, x_type, M, N, K)
            b = integers(fmt, N, K, ("tile", c))
            x = torch.randint(-8, 9, (M, K), device=DEV).to(TYPES[x_type])
            y = torch.full((M, N), float("nan"), device=DEV)
            run_linear(fmt, pack(fmt, b), x, y, M, N, K)
            assert np.array_equal(f64(y), f64(x) @ _linref.dequantize(fmt, b).T)


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("fmt", FMTS)
def test_every_tile_in_groups(fmt, x_type):
    """Groups from none to three times the mean, so that a tile's whole rows and short ends both run."""
    N, E = 1030, 40
    for c, mean in sorted(grouped_shapes(fmt, x_type).items()):
        for K in (64, 288):
            say("groups", c, fmt, x_type, mean, K)
            g = np.random.default_rng(mean)
            cut = np.sort(np.concatenate([[0], g.integers(0, mean * E + 1, E // 2 - 1).repeat(2), [0, mean * E]]))
            off = torch.from_numpy(cut.astype(np.int32)).to(DEV)
            R = mean * E
            b = integers(fmt, E * N, K, ("groups", c))
            W = _linref.dequantize(fmt, b).reshape(E, N, K)
            x = torch.randint(-8, 9, (R, K), device=DEV).to(TYPES[x_type])
            y = torch.full((R, N), float("nan"), device=DEV)
            run_grouped(fmt, pack(fmt, b), E, off, x, y, R, N, K)
            got, xs = f64(y), f64(x)
            for e in range(E):
                i, j = cut[e], cut[e + 1]
                assert np.array_equal(got[i:j], xs[i:j] @ W[e].T), f"group {e}"


@pytest.mark.parametrize("M,N", [(70, 4099), (300, 4099), (600, 4099), (300, 8195)])
@pytest.mark.parametrize("nb", [1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 13, 16, 17, 33])
def test_every_length_of_k(nb, M, N):
    """From one block on: the steps of 64 come in fours, an odd block last."""
    K = nb * 32
    for fmt in FMTS:
        say("length", nb, M, N, fmt)
        b = _linref.blocks(fmt, 40, K, ("len",))
        wide = np.ascontiguousarray(np.tile(b, (N // 40 + 1, 1, 1))[:N])
        x, y = rows(M, K, ("len-x", M), torch.bfloat16), torch.empty((M, N), device=DEV)
        run_linear(fmt, pack(fmt, wide), x, y, M, N, K)
        check(y[:, :40], _linref.dequantize(fmt, b), x, K, torch.float32, f"{fmt} {nb}")
        whole = y[:, :N // 40 * 40].reshape(M, -1, 40)
        assert torch.equal(whole, whole[:, :1].expand_as(whole))  # the same rows of weights give the same bits


@pytest.mark.parametrize("x_type", ["bf16", "f32"])
def test_mxfp4_scales_at_both_ends(x_type):
    """Blocks whose largest weights pass 2^127, NaN scales and the lowest scale, in tiles and in their last rows."""
    K = 128
    for M, N in ((70, 4099), (600, 4099)):
        say("scales", x_type, M, N)
        b = _linref.blocks("mxfp4", N, K, ("ends",))
        b[5, 1, 0], b[5, 0, 0] = 254, 253
        b[4098, 3, 0] = 254
        b[1000, 2, 0] = 255
        b[77, :, 0] = 0
        W = _linref.dequantize("mxfp4", b)
        x = (rows(M, K, ("ends-x", M), torch.float32) * 2.0 ** -20).to(TYPES[x_type])
        y = torch.empty((M, N), device=DEV)
        run_linear("mxfp4", pack("mxfp4", b), x, y, M, N, K)
        Y, S = _linref.linear(W, f64(x))
        tol = _linref.tolerance(Y, S, K, torch.float32) + 2.0 ** -133 * np.nansum(np.abs(W), 1)
        _linref.close(f64(y), Y, tol, f"{x_type} {M}")


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("M,N", [(70, 4099), (600, 4099)])
def test_infinities_and_nan_in_tiles(M, N, x_type):
    """They go as far as the formula takes them: to their row of x, or to the weight row of a scale."""
    K = 160
    for fmt in FMTS:
        say("odd", fmt, x_type, M, N)
        b = _linref.blocks(fmt, N, K, ("odd-t",))
        if fmt == "q8_0":
            b[..., 2:] |= 1  # no code is 0, whose product with an infinity is NaN
        elif fmt == "q4_0":
            b[..., 2:] = np.where(b[..., 2:] & 15 == 8, b[..., 2:] | 1, b[..., 2:])
            b[..., 2:] = np.where(b[..., 2:] >> 4 == 8, b[..., 2:] | 16, b[..., 2:])
        else:
            b[..., 1:] |= 0x11
        x = rows(M, K, ("odd-tx", M), TYPES[x_type])
        x[0, 5] = float("inf")
        x[40, 100] = float("nan")
        x[M - 1, 159], x[M - 1, 3] = -float("inf"), float("inf")
        y = torch.empty((M, N), device=DEV)
        run_linear(fmt, pack(fmt, b), x, y, M, N, K)
        check(y, _linref.dequantize(fmt, b), x, K, torch.float32, f"{fmt} {x_type}")


@pytest.mark.parametrize("x_type", list(TYPES))
def test_empty_sum_in_tiles(x_type):
    for fmt in FMTS:
        say("K = 0", fmt, x_type)
        bias, y = gen.normal((4099,), ("k0t",), device=DEV), torch.empty((600, 4099), device=DEV)
        bqm.bqm_linear(fmt, None, torch.empty((600, 0), dtype=TYPES[x_type], device=DEV), 0, y, 4099, 600, 4099, 0, bias=bias, act="relu")
        assert torch.equal(y, bias.clamp(min=0).expand(600, 4099))


@pytest.mark.parametrize("M,N", [(70, 4099), (600, 4099), (600, 4100)])
def test_epilogue_and_edges_in_tiles(M, N):
    """Rows at strides that are multiples of four and that are not, in place, what lies around them kept."""
    K, out = 96, torch.bfloat16
    b = _linref.blocks("q8_0", N, K, ("epi-t",))
    W, wp = _linref.dequantize("q8_0", b), pack("q8_0", b)
    x, bias = rows(M, K, ("epi-tx",), out, pad=8), gen.normal((N,), ("epi-tb",), device=DEV)
    mul = rows(M, N, ("epi-tm",), out)
    for pad in (1, 5, 4 - N % 4):
        say("edges", M, N, pad)
        whole = torch.full((M + 2, N + pad), 7.0, dtype=out, device=DEV)
        inner = whole[1:M + 1, :N] if (N + pad) * 2 % 16 == 0 else whole[:M, :N]  # rows of Y start at a multiple of 16 bytes
        inner.copy_(gen.normal((M, N), ("epi-ty",), device=DEV))
        res = inner.clone()
        run_linear("q8_0", wp, x, inner, M, N, K, bias=bias, act="gelu_tanh", mul=mul, res=inner)
        check(inner, W, x, K, out, f"{M} {N} {pad}", bias=bias, act="gelu_tanh", mul=mul, res=res)
        assert (whole[:, N:] == 7.0).all() and (whole[M + 1:] == 7.0).all()


def test_graph_of_tiles():
    say("graph of tiles")
    M, N, K, E = 300, 4099, 288, 5
    b = _linref.blocks("mxfp4", N, K, ("g-t",))
    x, y, z = rows(M, K, ("g-tx",), torch.bfloat16), torch.empty((M, N), dtype=torch.bfloat16, device=DEV), torch.empty((M, 1030), device=DEV)
    be = _linref.blocks("q4_0", E * 1030, K, ("g-te",))
    off = torch.tensor([0, 150, 150, 151, 290, 300], dtype=torch.int32, device=DEV)
    wp, we = pack("mxfp4", b), pack("q4_0", be)

    def run():
        run_linear("mxfp4", wp, x, y, M, N, K, act="silu")
        run_grouped("q4_0", we, E, off, x, z, M, 1030, K)

    replays_match_eager(run, [y, z])

"""The linear layer, its grouped form and the embedding on the GPU, against the plain 64-bit forms of tests/_linref.py."""
import numpy as np
import pytest
import torch

import gen
from block_quantized_matrix_amd import bqm
from tests import _linref
from tests._gpu import DEV, host, say
from tests._linref import ACTS, FMTS, TYPES
from tests.test_gpu_graphs import replays_match_eager

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1, 32), (1, 40, 96), (3, 17, 160), (4, 200, 4096), (5, 100, 544), (16, 64, 1056), (17, 33, 128), (33, 1000, 4128),
          (64, 96, 512), (65, 257, 288), (130, 300, 1056), (300, 530, 1024)]


def pack(fmt, b):
    rows, nb = b.shape[:2]
    return bqm.repack(fmt, torch.from_numpy(b).to(DEV).reshape(-1), rows, nb * 32)


def rows(M, width, key, dtype, pad=0, fill=None):
    """M rows of normal numbers on the device, pad elements apart; what lies between them is `fill`."""
    t = gen.normal((M, width), key, device=DEV).to(dtype)
    if not pad:
        return t
    out = torch.full((M, width + pad), float("nan") if fill is None else fill, dtype=dtype, device=DEV)[:, :width]
    out.copy_(t)
    return out


def f64(t):
    return None if t is None else host(t.float()).astype(np.float64)


def run_linear(fmt, wp, x, y, M, N, K, bias=None, act="none", mul=None, res=None, **more):
    bqm.bqm_linear(fmt, wp, x, x.stride(0), y, y.stride(0), M, N, K, bias=bias, act=act, mul=mul,
                   mul_stride=0 if mul is None else mul.stride(0), residual=res, res_stride=0 if res is None else res.stride(0),
                   **more)


def run_grouped(fmt, wp, E, off, x, y, R, N, K, bias=None, act="none", mul=None, res=None, **more):
    bqm.bqm_linear_grouped(fmt, wp, E, off, x, x.stride(0), y, y.stride(0), R, N, K, bias=bias, act=act, mul=mul,
                           mul_stride=0 if mul is None else mul.stride(0), residual=res,
                           res_stride=0 if res is None else res.stride(0), **more)


def check(got, W, x, K, out, what, bias=None, act="none", mul=None, res=None):
    y, S = _linref.linear(W, f64(x), f64(bias), act, f64(mul), f64(res))
    _linref.close(f64(got), y, _linref.tolerance(y, S, K, out, f64(mul), f64(res)), what)


# ---- one matrix ----

@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_matches_definition(M, N, K, fmt, x_type):
    say("linear", fmt, x_type, M, N, K)
    b = _linref.blocks(fmt, N, K, ("w",))
    x, y = rows(M, K, ("lin-x", M, K), TYPES[x_type]), torch.empty((M, N), device=DEV)
    run_linear(fmt, pack(fmt, b), x, y, M, N, K)
    check(y, _linref.dequantize(fmt, b), x, K, torch.float32, f"{fmt} {x_type} {M} {N} {K}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("y_type", list(TYPES))
@pytest.mark.parametrize("M", [1, 7, 40, 200])
def test_linear_epilogue(M, y_type, act):
    """Every activation and type with bias, mul and residual, each alone and together; rows apart, what lies between them kept."""
    N, K, fmt = 150, 256, "q8_0"
    b = _linref.blocks(fmt, N, K, ("epi",))
    W, wp, out = _linref.dequantize(fmt, b), pack(fmt, b), TYPES[y_type]
    x = rows(M, K, ("epi-x", M), torch.bfloat16, pad=8)
    bias = gen.normal((N,), ("epi-b",), device=DEV)
    mul, res = rows(M, N, ("epi-m", M), out, pad=3), rows(M, N, ("epi-r", M), out, pad=10)
    for mask in range(8):
        say("epilogue", M, y_type, act, mask)
        more = dict(bias=bias if mask & 1 else None, mul=mul if mask & 2 else None, res=res if mask & 4 else None, act=act)
        whole = torch.full((M, N + 5), 7.0, dtype=out, device=DEV)
        run_linear(fmt, wp, x, whole[:, :N], M, N, K, **more)
        check(whole[:, :N], W, x, K, out, f"{y_type} {act} {mask}", **more)
        assert (whole[:, N:] == 7.0).all()


@pytest.mark.parametrize("M", [2, 100])
def test_linear_in_place(M):
    """mul and residual may be Y itself."""
    N, K, fmt = 96, 128, "mxfp4"
    b = _linref.blocks(fmt, N, K, ("inpl",))
    W, wp, x = _linref.dequantize(fmt, b), pack(fmt, b), rows(M, K, ("inpl-x",), torch.float16)
    for which in ("mul", "res"):
        say("in place", M, which)
        y = rows(M, N, ("inpl-y",), torch.float16)
        before = y.clone()
        run_linear(fmt, wp, x, y, M, N, K, act="silu", **{which: y})
        check(y, W, x, K, torch.float16, which, act="silu", **{which: before})


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("x_type", list(TYPES))
def test_linear_exact_on_integers(fmt, x_type):
    """Small integers and scales that are powers of two leave nothing to round: any wrong code, scale or place shows."""
    for M, N, K in ((1, 300, 1056), (16, 50, 4096), (70, 260, 544), (260, 300, 1024)):
        say("integers", fmt, x_type, M, N, K)
        b = _linref.blocks(fmt, N, K, ("int", M))
        g = np.random.default_rng(M)
        if fmt == "mxfp4":
            b[..., 0] = g.integers(126, 129, (N, K // 32))
        else:
            b[..., :2] = g.choice(np.array([0.5, 1, 2, -1], np.float16), (N, K // 32))[..., None].view(np.uint8)
            if fmt == "q8_0":
                b[..., 2:] = g.integers(-9, 10, (N, K // 32, 32)).astype(np.int8).view(np.uint8)
        x = torch.randint(-8, 9, (M, K), device=DEV).to(TYPES[x_type])
        y = torch.empty((M, N), device=DEV)
        run_linear(fmt, pack(fmt, b), x, y, M, N, K)
        assert np.array_equal(f64(y), f64(x) @ _linref.dequantize(fmt, b).T)


@pytest.mark.parametrize("M", [1, 40, 150])
def test_linear_empty_sum(M):
    """K = 0: the sum is 0 and the rest is done."""
    say("K = 0", M)
    bias, y = gen.normal((50,), ("k0",), device=DEV), torch.empty((M, 50), device=DEV)
    bqm.bqm_linear("q4_0", None, torch.empty((M, 0), device=DEV), 0, y, 50, M, 50, 0, bias=bias, act="relu")
    assert torch.equal(y, bias.clamp(min=0).expand(M, 50))


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("M", [3, 50, 140])
def test_linear_infinities_and_nan(M, x_type):
    """An infinity or a NaN in a row or a scale goes as far as the formula takes it and no further."""
    N, K = 70, 160
    for fmt in FMTS:
        say("odd", fmt, x_type, M)
        b = _linref.blocks(fmt, N, K, ("odd",))
        if fmt == "q8_0":
            b[..., 2:] |= 1  # no code is 0, whose product with an infinity is NaN
        elif fmt == "q4_0":
            b[..., 2:] = np.where(b[..., 2:] & 15 == 8, b[..., 2:] | 1, b[..., 2:])
            b[..., 2:] = np.where(b[..., 2:] >> 4 == 8, b[..., 2:] | 16, b[..., 2:])
        else:
            b[..., 1:] |= 0x11
            b[7, 2, 0] = 255
        W = _linref.dequantize(fmt, b)
        x = rows(M, K, ("odd-x", M), TYPES[x_type])
        x[0, 5] = float("inf")
        x[1, 100] = float("nan")
        x[2, 159], x[2, 3] = -float("inf"), float("inf")
        y = torch.empty((M, N), device=DEV)
        run_linear(fmt, pack(fmt, b), x, y, M, N, K)
        check(y, W, x, K, torch.float32, f"{fmt} {x_type}")


def test_linear_payload_nan():
    """A NaN of fp32 whose upper half alone would be an infinity."""
    say("payload")
    b = _linref.blocks("q8_0", 20, 64, ("pay",))
    for M in (2, 80):
        x = rows(M, 64, ("pay-x",), torch.float32)
        x.view(torch.int32)[1, 9] = 0x7F800001
        y = torch.empty((M, 20), device=DEV)
        run_linear("q8_0", pack("q8_0", b), x, y, M, 20, 64)
        y = host(y)
        assert np.isnan(y[1]).all() and np.isfinite(np.delete(y, 1, 0)).all()


@pytest.mark.parametrize("M", [2, 100])
def test_linear_far_numbers(M):
    """The smallest and largest numbers: subnormal fp16 and fp32 rows, scales at both ends of e8m0, subnormal d."""
    say("far", M)
    N, K = 40, 96
    for x_type, size in (("f16", 2.0 ** -20), ("f32", 2.0 ** -122), ("bf16", 2.0 ** -120), ("f32", 2.0 ** 100)):
        for fmt in FMTS:
            b = _linref.blocks(fmt, N, K, ("far",))
            if fmt == "mxfp4":
                b[..., 0] = np.where(b[..., 0] > 119, 254 if size < 1 else 3, 127)
            else:
                b[:20, :, :2] = np.array([5e-7 if size > 1 else 60000.0], np.float16).view(np.uint8)
            x = (gen.normal((M, K), ("far-x",), device=DEV) * size).to(TYPES[x_type])
            y = torch.empty((M, N), device=DEV)
            run_linear(fmt, pack(fmt, b), x, y, M, N, K)
            W = _linref.dequantize(fmt, b)
            Y, S = _linref.linear(W, f64(x))
            tol = _linref.tolerance(Y, S, K, torch.float32)
            if x_type == "f32":  # what is below the resolution of the parts
                tol = tol + 2.0 ** -133 * np.abs(W).sum(1)
            _linref.close(f64(y), Y, tol, f"{fmt} {x_type} {size}")


# ---- matrices of experts ----

GROUPS = [
    [0, 1], [0, 5], [0, 0, 0, 3], [0, 1, 2, 3, 4], [0, 17, 17, 18, 50, 50], [2, 9, 9, 40], [0, 130, 131, 131, 131, 400, 401],
    [0, 64, 128, 192], [0, 200, 200, 200]]


@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("off", GROUPS)
@pytest.mark.parametrize("N,K", [(50, 160), (264, 1024)])
def test_grouped_matches_definition(N, K, off, fmt, x_type):
    """Groups of any length, also none; rows before the first and behind the last group are left as they were."""
    say("grouped", off, fmt, x_type, N, K)
    E, R, out = len(off) - 1, off[-1] + 3, TYPES[x_type]
    b = _linref.blocks(fmt, E * N, K, ("grp", E))
    W = _linref.dequantize(fmt, b)
    x, bias = rows(R, K, ("grp-x", R, K), out, pad=16), gen.normal((E, N), ("grp-b", E), device=DEV)
    mul, res = rows(R, N, ("grp-m", R), out), rows(R, N, ("grp-r", R), out, pad=1)
    y = torch.full((R, N), 5.0, dtype=out, device=DEV)
    run_grouped(fmt, pack(fmt, b), E, torch.tensor(off, dtype=torch.int32, device=DEV), x, y, R, N, K, bias=bias, act="gelu", mul=mul,
                res=res)
    for e, (i, j) in enumerate(zip(off, off[1:])):
        if j > i:
            check(y[i:j], W[e * N:(e + 1) * N], x[i:j], K, out, f"group {e}", bias=bias[e], act="gelu", mul=mul[i:j], res=res[i:j])
    assert (y[:off[0]] == 5.0).all() and (y[off[-1]:] == 5.0).all()


def test_grouped_many_experts():
    """More experts than a workgroup has threads, most of them without rows."""
    E, N, K, R = 3000, 8, 64, 700
    say("grouped", E)
    counts = torch.bincount(torch.from_numpy(np.random.default_rng(3).integers(0, 600, R) * 5), minlength=E)
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    b = _linref.blocks("q4_0", E * N, K, ("many",))
    W = _linref.dequantize("q4_0", b).reshape(E, N, K)
    x, y = rows(R, K, ("many-x",), torch.bfloat16), torch.empty((R, N), device=DEV)
    run_grouped("q4_0", pack("q4_0", b), E, off.to(torch.int32).to(DEV), x, y, R, N, K)
    which = torch.repeat_interleave(torch.arange(E), counts).numpy()
    xs = f64(x)
    Y, S = np.einsum("rk,rnk->rn", xs, W[which]), np.einsum("rk,rnk->rn", np.abs(xs), np.abs(W[which]))
    _linref.close(f64(y), Y, _linref.tolerance(Y, S, K, torch.float32), "many experts")


@pytest.mark.parametrize("off", [[0, 4, 1 << 30], [-5, 4, 9], [0, 9, 2], [9, 3, 20], [-(1 << 31), -1, (1 << 31) - 1]])
def test_grouped_offsets_out_of_range(off):
    """Whatever the offsets hold, nothing outside Y's rows is written; in order, they count as 0 or R beyond the ends."""
    say("offsets", off)
    E, N, K, R = 2, 40, 64, 9
    b = _linref.blocks("q8_0", E * N, K, ("oor",))
    W = _linref.dequantize("q8_0", b)
    x = rows(R, K, ("oor-x",), torch.float32)
    whole = torch.full((R + 40, N), 3.0, device=DEV)
    y = whole[20:20 + R]
    run_grouped("q8_0", pack("q8_0", b), E, torch.tensor(off, dtype=torch.int32, device=DEV), x, y, R, N, K)
    assert (whole[:20] == 3.0).all() and (whole[20 + R:] == 3.0).all()
    if off == sorted(off):
        o = [min(max(v, 0), R) for v in off]
        for e in range(E):
            if o[e + 1] > o[e]:
                check(y[o[e]:o[e + 1]], W[e * N:(e + 1) * N], x[o[e]:o[e + 1]], K, torch.float32, f"group {e}")


# ---- a table's rows ----

@pytest.mark.parametrize("y_type", list(TYPES))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,K", [(1, 32), (1, 4096), (5, 160), (70, 544), (300, 1056)])
def test_embed_matches_definition(T, K, fmt, y_type):
    n, out = 50, TYPES[y_type]
    b = _linref.blocks(fmt, n, K, ("emb",))
    W, wp = _linref.dequantize(fmt, b), pack(fmt, b)
    ids = torch.from_numpy(np.random.default_rng(T).integers(0, n, T).astype(np.int32)).to(DEV)
    for scale, pad in ((1.0, 0), (0.1, 3), (22.5, 8)):
        say("embed", fmt, y_type, T, K, scale, pad)
        whole = torch.full((T, K + pad), 9.0, dtype=out, device=DEV)
        bqm.bqm_embed(fmt, wp, n, K, ids, T, scale, whole, K + pad)
        want = W[host(ids)] * np.float64(np.float32(scale))
        f = torch.finfo(out)  # the product in fp32, then the type: half a step each
        _linref.close(f64(whole[:, :K]), want, np.abs(want) * (f.eps / 2 + 2.0 ** -24) * 1.01 + f.tiny * f.eps / 2, f"{fmt} {y_type}")
        assert (whole[:, K:] == 9.0).all()


@pytest.mark.parametrize("y_type", list(TYPES))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,K", [(3300, 2592), (16500, 96)])
def test_embed_many_rows(T, K, fmt, y_type):
    """Calls large enough for several runs a wave, the last of a row short or absent."""
    say("embed many", fmt, y_type, T, K)
    n, out = 40, TYPES[y_type]
    b = _linref.blocks(fmt, n, K, ("emb-m",))
    wp = pack(fmt, b)
    ids = torch.from_numpy(np.random.default_rng(T).integers(-2, n + 2, T).astype(np.int32)).to(DEV)
    W = torch.from_numpy(_linref.dequantize(fmt, b)).to(DEV)
    table = torch.cat([torch.zeros((2, K), dtype=torch.float64, device=DEV), W, torch.full((2, K), float("nan"), dtype=torch.float64, device=DEV)])
    want = table[ids.long() + 2] * float(np.float32(0.1))
    f = torch.finfo(out)  # the product in fp32, then the type: half a step each
    most = want.abs() * (f.eps / 2 + 2.0 ** -24) * 1.01 + f.tiny * f.eps / 2
    inside = (ids >= 0) & (ids < n)
    for pad in (0, 3, 8):
        whole = torch.full((T + 1, K + pad), 9.0, dtype=out, device=DEV)
        bqm.bqm_embed(fmt, wp, n, K, ids, T, 0.1, whole, K + pad)
        y = whole[:T, :K].double()
        assert ((y - want).abs() <= most)[inside].all()
        assert (y[ids < 0] == 0).all() and y[ids >= n].isnan().all()
        assert (whole[:T, K:] == 9.0).all() and (whole[T] == 9.0).all()


def test_embed_ids_outside():
    """Negative ids give zeros, ids past the table NaN; an empty table has no ids inside."""
    say("embed ids")
    n, K = 20, 96
    b = _linref.blocks("q4_0", n, K, ("emb-o",))
    W = _linref.dequantize("q4_0", b)
    ids = torch.tensor([3, -1, 19, 20, -(1 << 31), (1 << 31) - 1, 0, 3], dtype=torch.int32, device=DEV)
    y = torch.empty((8, K), device=DEV)
    bqm.bqm_embed("q4_0", pack("q4_0", b), n, K, ids, 8, 1.0, y, K)
    y = f64(y)
    for t, i in enumerate(host(ids)):
        want = np.zeros(K) if i < 0 else np.full(K, np.nan) if i >= n else W[i]
        assert np.array_equal(y[t], want, equal_nan=True)
    z = torch.empty((8, K), device=DEV)
    bqm.bqm_embed("q4_0", None, 0, K, ids, 8, 1.0, z, K)
    assert (z[ids < 0] == 0).all() and z[ids >= 0].isnan().all()


def test_embed_mxfp4_scales():
    """Every scale byte; a weight beyond fp32's range under a scale that brings it back."""
    say("embed scales")
    b = np.zeros((256, 1, 17), np.uint8)
    b[:, 0, 0] = np.arange(256)
    b[:, 0, 1:] = np.arange(16) | np.arange(16)[::-1] << 4
    W, wp = _linref.dequantize("mxfp4", b), pack("mxfp4", b)
    ids = torch.arange(256, dtype=torch.int32, device=DEV)
    for scale in (1.0, 0.25, 2.0 ** -20):
        y = torch.empty((256, 32), device=DEV)
        bqm.bqm_embed("mxfp4", wp, 256, 32, ids, 256, scale, y, 32)
        with np.errstate(over="ignore"):
            want = (W * scale).astype(np.float32)
        assert np.array_equal(host(y), want, equal_nan=True)


# ---- as they are used ----

def test_far_offsets():
    """Rows of x and y, and an expert's matrix, that begin more than 2^31 bytes after the first."""
    say("far offsets")
    R, S, N, K = 1100, 1 << 20, 48, 64
    b = _linref.blocks("q8_0", N, K, ("off",))
    W, wp = _linref.dequantize("q8_0", b), pack("q8_0", b)
    x = torch.zeros((R, S), dtype=torch.bfloat16, device=DEV)[:, :K]
    x.copy_(gen.normal((R, K), ("off-x",), device=DEV))
    y = torch.zeros((R, S), dtype=torch.bfloat16, device=DEV)[:, :N]
    run_linear("q8_0", wp, x, y, R, N, K)
    check(y, W, x, K, torch.bfloat16, "far rows")
    del x, y
    E, N, K = 3, 300000, 4096  # 1.2 GB of codes each
    room = torch.zeros(bqm.packed_bytes("q8_0", E * N, K), dtype=torch.uint8, device=DEV)
    nb, last = K // 32, E * N - 1
    b = _linref.blocks("q8_0", 1, K, ("off-w",))
    room[last * K:(last + 1) * K] = torch.from_numpy(b[..., 2:].reshape(-1)).to(DEV)
    room[E * N * K + last * nb * 2:E * N * K + (last + 1) * nb * 2] = torch.from_numpy(b[..., :2].reshape(-1)).to(DEV)
    for M in (1, 70):
        x, y = rows(M, K, ("off-x2",), torch.bfloat16), torch.empty((M, N), device=DEV)
        off = torch.tensor([0, 0, 0, M], dtype=torch.int32, device=DEV)
        run_grouped("q8_0", room, E, off, x, y, M, N, K)
        check(y[:, -1:], _linref.dequantize("q8_0", b), x, K, torch.float32, "far expert")
        assert (y[:, :-1] == 0).all()


def test_on_another_stream_and_deterministic():
    say("streams")
    N, K = 500, 1056
    for M in (3, 40, 200):
        b = _linref.blocks("q4_0", N, K, ("str",))
        wp, x = pack("q4_0", b), rows(M, K, ("str-x",), torch.bfloat16)
        torch.cuda.synchronize()
        got = []
        for s in (torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.current_stream()):
            y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
            s.wait_stream(torch.cuda.current_stream())
            run_linear("q4_0", wp, x, y, M, N, K, stream=s)
            got.append(y)
        torch.cuda.synchronize()
        assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("T", [2, 60])
def test_a_layer_from_ids_to_rows(T):
    """Embedding, a gated feed-forward with its residual, a router and its experts' gated feed-forward, captured and replayed:
    each step against the plain form of its own inputs."""
    say("layer", T)
    V, H, F, E, FE, top_k = 90, 256, 544, 6, 96, 2
    fmt = {"tab": "q8_0", "gate": "q4_0", "up": "q4_0", "down": "mxfp4", "eg": "q4_0", "eu": "q8_0", "ed": "mxfp4"}
    shape = {"tab": (V, H), "gate": (F, H), "up": (F, H), "down": (H, F), "eg": (E * FE, H), "eu": (E * FE, H), "ed": (E * H, FE)}
    blk = {n: _linref.blocks(fmt[n], *shape[n], ("layer", n)) for n in fmt}
    W = {n: _linref.dequantize(fmt[n], blk[n]) for n in fmt}
    wp = {n: pack(fmt[n], blk[n]) for n in fmt}
    bf = torch.bfloat16
    ids = torch.from_numpy(np.random.default_rng(T).integers(0, V, T).astype(np.int32)).to(DEV)
    wr = gen.normal((H, E), ("layer-r",), device=DEV)
    R = T * top_k
    h0, up, mid, h1 = (torch.empty((T, w), dtype=bf, device=DEV) for w in (H, F, F, H))
    eids, ew = torch.empty((T, top_k), dtype=torch.int32, device=DEV), torch.empty((T, top_k), device=DEV)
    logits = torch.empty((T, E), device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    xs, eu, em, ey = (torch.empty((R, w), dtype=bf, device=DEV) for w in (H, FE, FE, H))

    def dense():
        bqm.bqm_embed(fmt["tab"], wp["tab"], V, H, ids, T, 16.0, h0, H)
        run_linear(fmt["up"], wp["up"], h0, up, T, F, H)
        run_linear(fmt["gate"], wp["gate"], h0, mid, T, F, H, act="silu", mul=up)
        run_linear(fmt["down"], wp["down"], mid, h1, T, H, F, res=h0)

    def experts():
        run_grouped(fmt["eu"], wp["eu"], E, off, xs, eu, R, FE, H)
        run_grouped(fmt["eg"], wp["eg"], E, off, xs, em, R, FE, H, act="silu", mul=eu)
        run_grouped(fmt["ed"], wp["ed"], E, off, em, ey, R, H, FE)

    replays_match_eager(dense, [h0, up, mid, h1])
    torch.mm(h1.float(), wr, out=logits)
    bqm.bqm_route("softmax", logits, E, None, T, E, 1, 1, 1, top_k, True, 1.0, eids, ew)
    flat = eids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    off[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    xs.copy_(h1[order // top_k])
    replays_match_eager(experts, [eu, em, ey])
    assert np.abs(f64(h0) - W["tab"][host(ids)] * 16).max() <= 2.0 ** -8 * np.abs(f64(h0)).max()
    check(up, W["up"], h0, H, bf, "up")
    check(mid, W["gate"], h0, H, bf, "gate", act="silu", mul=up)
    check(h1, W["down"], mid, F, bf, "down", res=h0)
    o = host(off)
    assert o[-1] == R
    for e in range(E):
        i, j = o[e], o[e + 1]
        if j > i:
            check(eu[i:j], W["eu"][e * FE:(e + 1) * FE], xs[i:j], H, bf, "expert up")
            check(em[i:j], W["eg"][e * FE:(e + 1) * FE], xs[i:j], H, bf, "expert gate", act="silu", mul=eu[i:j])
            check(ey[i:j], W["ed"][e * H:(e + 1) * H], em[i:j], FE, bf, "expert down")

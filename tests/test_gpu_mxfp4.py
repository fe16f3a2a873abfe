"""MXFP4 on the GPU: quantizer, repacking, the decode and prefill products and the expert-indexed one, against the plain
64-bit forms of tests/_mxref.py."""
import numpy as np
import pytest
import torch

import gen
from block_quantized_matrix_amd import bqm
from tests import _mxref
from tests._gpu import DEV, host, say
from tests.test_gpu_graphs import replays_match_eager

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def room(rows, K, fill=0xA5):
    return torch.full((bqm.packed_bytes("mxfp4", rows, K),), fill, dtype=torch.uint8, device=DEV)


def quantized(x):
    rows, K = x.shape
    p = room(rows, K)
    bqm.bqm_quantize_mxfp4(x, x.stride(0), p, rows, K)
    return p


def unpacked(p, rows, K):
    out = torch.full((rows, K // 32, 17), 0xEE, dtype=torch.uint8, device=DEV)
    bqm.bqm_unpack("mxfp4", p, out, rows, K)
    return out


def blocks(rows, K, key, lo=118, hi=132):
    """Random interchange blocks: every code, scale bytes in [lo, hi]."""
    g = np.random.default_rng(gen.seed_of(*key))
    b = g.integers(0, 256, (rows, K // 32, 17), dtype=np.uint8)
    b[..., 0] = g.integers(lo, hi + 1, (rows, K // 32))
    return b


def packed(b):
    rows, nb = b.shape[:2]
    p = room(rows, nb * 32)
    bqm.bqm_repack("mxfp4", torch.from_numpy(b).to(DEV), p, rows, nb * 32)
    return p


def close(y, Y, S, K, what):
    """|y - Y| <= tolerance(K) S where Y is a number, NaN exactly where Y is NaN."""
    y = np.asarray(y, np.float64)
    nan = np.isnan(Y)
    assert np.array_equal(np.isnan(y), nan), f"{what}: NaN in other places"
    err = np.where(nan, 0, np.abs(np.where(nan, 0, y) - np.where(nan, 0, Y)))
    bad = err > _mxref.tolerance(K) * np.where(nan, 0, S)
    assert not bad.any(), f"{what}: {int(bad.sum())} outputs off, worst {np.max(err / np.maximum(S, 1e-300))} of S"


# ---- quantizer and layout ----

@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (16, 128), (17, 544), (33, 1056), (250, 4128)])
def test_quantize_matches_definition(dtype, rows, K):
    say("quantize", dtype, rows, K)
    x = gen.normal((rows, K), ("mxq", rows, K), device=DEV)
    x = (x * torch.exp2(torch.randint(-12, 12, (rows, K), device=DEV).float())).to(TYPES[dtype])
    p = quantized(x)
    want = _mxref.quantize(host(x.float()))
    assert np.array_equal(host(unpacked(p, rows, K)), want)
    # the padding too is written: repacking the same blocks gives the same buffer
    assert torch.equal(packed(want), p)


def test_quantize_edges():
    say("quantize edges")
    t = 2.0 ** np.arange(-149, 128)
    x = np.zeros((40, 64), np.float32)
    x[0, :7] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    x[0, 31] = 6.0
    x[1, :7] = -x[0, :7]
    x[1, 31] = 7.99
    x[2, 3] = -0.0                                    # a block of zeros keeps the sign of zero in the code
    x[3, 5], x[3, 40] = np.inf, np.nan
    x[4, 0], x[4, 33] = -np.inf, 1.0
    x[5, :] = np.float32(3.4028235e38)                # the largest finite value
    x[6, :32] = np.float32(1.4e-45)                   # the smallest
    x[7, :32] = (2.0 ** np.arange(-149, -117))
    for r in range(8, 40):
        x[r] = np.resize(t[(r - 8) * 8:], 64)
    xd = torch.from_numpy(x).to(DEV)
    assert np.array_equal(host(unpacked(quantized(xd), 40, 64)), _mxref.quantize(x))


def test_quantize_strides_and_offsets():
    """Rows apart, rows that start at odd elements, and no read or write between them."""
    say("quantize strides")
    for dtype in TYPES.values():
        for stride, K in ((97, 96), (160, 128), (1000, 992)):
            flat = gen.normal((21 * stride,), ("mxs", stride), device=DEV).to(dtype)
            x = flat.as_strided((21, K), (stride, 1))
            p = quantized(x)
            assert np.array_equal(host(unpacked(p, 21, K)), _mxref.quantize(host(x.float())))
            y = torch.full((21, stride), 7.0, dtype=dtype, device=DEV)
            bqm.bqm_dequantize_mxfp4(p, y, stride, 21, K)
            got = host(y.float())
            want = torch.from_numpy(_mxref.dequantize(_mxref.quantize(host(x.float())))).to(dtype)
            assert np.array_equal(got[:, :K], want.float().numpy()) and (got[:, K:] == 7.0).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_dequantize_every_code_and_scale(dtype):
    say("dequantize", dtype)
    b = np.zeros((256, 1, 17), np.uint8)
    b[:, 0, 0] = np.arange(256)
    b[:, 0, 1:] = np.arange(16) | np.arange(16)[::-1] << 4
    y = torch.empty((256, 32), dtype=TYPES[dtype], device=DEV)
    bqm.bqm_dequantize_mxfp4(packed(b), y, 32, 256, 32)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(_mxref.dequantize(b)).to(TYPES[dtype]).float().numpy()
    assert np.array_equal(host(y.float()), want, equal_nan=True)


@pytest.mark.parametrize("rows,K", [(1, 32), (5, 160), (47, 640), (128, 1024)])
def test_repack_round_trip_unaligned(rows, K):
    say("repack", rows, K)
    b = blocks(rows, K, ("mxr", rows), 0, 255)
    raw = torch.zeros(b.size + 3, dtype=torch.uint8, device=DEV)
    raw[3:] = torch.from_numpy(b).to(DEV).reshape(-1)
    p = room(rows, K)
    bqm.bqm_repack("mxfp4", raw.data_ptr() + 3, p, rows, K)
    assert np.array_equal(host(unpacked(p, rows, K)), b)


# ---- decode product ----

@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("N,K", [(1, 32), (15, 64), (16, 128), (130, 544), (517, 4096), (2000, 1056), (77, 17408)])
def test_qmv(M, N, K):
    say("qmv_mxfp4", M, N, K)
    b = blocks(N, K, ("mxv", N, K))
    X = gen.normal((M, K), ("mxv-x", M, K))
    Y = torch.full((M * N + 64,), 7.0, device=DEV)
    bqm.qmv_mxfp4(packed(b), X.to(DEV), Y, M, N, K)
    got = host(Y)
    assert (got[M * N:] == 7.0).all()
    close(got[:M * N].reshape(M, N), *_mxref.product(_mxref.dequantize(b), X.numpy().astype(np.float64)), K, "qmv")


def test_qmv_many_rows():
    """More rows than one round of workgroups takes, and a batch whose inputs do not fit local memory at once."""
    for M, N, K in ((1, 70001, 64), (8, 40000, 256), (8, 300, 32768), (1, 33, 65536)):
        say("qmv_mxfp4", M, N, K)
        b = blocks(N, K, ("mxm", N, K))
        X = gen.normal((M, K), ("mxm-x", M, K))
        Y = torch.empty((M, N), device=DEV)
        bqm.qmv_mxfp4(packed(b), X.to(DEV), Y, M, N, K)
        close(host(Y), *_mxref.product(_mxref.dequantize(b), X.numpy().astype(np.float64)), K, "qmv")


@pytest.mark.parametrize("M", [1, 4, 8])
def test_qmv_wide_inputs(M):
    """Inputs of very different sizes inside a block, the large ones against zero codes: the error stays relative to
    what is summed."""
    say("qmv wide", M)
    N, K = 64, 1024
    b = blocks(N, K, ("mxw",))
    X = gen.normal((M, K), ("mxw-x", M)).double().numpy() * 2.0 ** np.random.default_rng(1).integers(-30, 30, (M, K))
    X = X.astype(np.float32)
    W = _mxref.dequantize(b)
    big = np.abs(X).max(0) > 1e3
    codes = np.concatenate([b[..., 1:] & 15, b[..., 1:] >> 4], -1).reshape(N, K)
    codes[:, big] = 0
    c = codes.reshape(N, K // 32, 32)
    b[..., 1:] = c[..., :16] | c[..., 16:] << 4
    W = _mxref.dequantize(b)
    Y = torch.empty((M, N), device=DEV)
    bqm.qmv_mxfp4(packed(b), torch.from_numpy(X).to(DEV), Y, M, N, K)
    close(host(Y), *_mxref.product(W, X.astype(np.float64)), K, "qmv wide")


@pytest.mark.parametrize("M", [1, 8])
def test_qmv_exact_and_special(M):
    say("qmv special", M)
    N, K = 100, 768
    b = blocks(N, K, ("mxe",), 126, 128)
    X = gen.small_int((M, K), ("mxe-x", M))
    Y = torch.empty((M, N), device=DEV)
    run = lambda: bqm.qmv_mxfp4(packed(b), X.to(DEV), Y, M, N, K)  # noqa: E731
    run()
    assert np.array_equal(host(Y), (X.numpy().astype(np.float64) @ _mxref.dequantize(b).T).astype(np.float32))
    b[5, 3, 0] = 255  # a NaN scale makes its row NaN and no other
    run()
    got = host(Y)
    assert np.isnan(got[:, 5]).all() and np.isfinite(np.delete(got, 5, 1)).all()
    b[5, 3, 0] = 127
    X[M - 1, 40] = float("nan")  # a NaN input makes its output row NaN and no other
    run()
    got = host(Y)
    assert np.isnan(got[M - 1]).all() and np.isfinite(got[:M - 1]).all()
    X[M - 1, 40] = float("inf")
    run()
    got, w = host(Y)[M - 1], _mxref.dequantize(b)[:, 40]
    assert not np.isfinite(got).any()
    assert (got[w > 0] == np.inf).all() and (got[w < 0] == -np.inf).all() and np.isnan(got[w == 0]).all()


@pytest.mark.parametrize("lo,hi", [(0, 3), (250, 252)])
def test_qmv_extreme_scales(lo, hi):
    say("qmv scales", lo, hi)
    N, K = 48, 256
    b = blocks(N, K, ("mxx", lo), lo, hi)
    X = (gen.normal((2, K), ("mxx-x",)) * (2.0 ** 60 if lo == 0 else 2.0 ** -60)).float()
    Y = torch.empty((2, N), device=DEV)
    bqm.qmv_mxfp4(packed(b), X.to(DEV), Y, 2, N, K)
    close(host(Y), *_mxref.product(_mxref.dequantize(b), X.numpy().astype(np.float64)), K, "qmv scales")


def test_qmv_empty_sum_and_streams():
    say("qmv K = 0, and two streams at once")
    Y = torch.full((3, 50), 5.0, device=DEV)
    bqm.qmv_mxfp4(None, None, Y, 3, 50, 0)
    assert (host(Y) == 0).all()
    N, K = 1000, 2048
    b = [blocks(N, K, ("mxt", i)) for i in range(2)]
    p = [packed(v) for v in b]
    X = [gen.normal((8, K), ("mxt-x", i), device=DEV) for i in range(2)]
    out = [torch.empty((8, N), device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            bqm.qmv_mxfp4(p[i], X[i], out[i], 8, N, K, stream=streams[i])
    for i in range(2):
        close(host(out[i]), *_mxref.product(_mxref.dequantize(b[i]), host(X[i]).astype(np.float64)), K, "streams")


# ---- prefill product ----

@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 200, 4096), (5, 17, 160), (16, 16, 128), (33, 1000, 4128), (64, 128, 512),
                                   (100, 130, 544), (129, 257, 1056), (300, 513, 96), (512, 640, 2048), (1000, 96, 256),
                                   (260, 2050, 640)])
def test_qmm(M, N, K):
    say("qmm_mxfp4", M, N, K)
    w, x = blocks(N, K, ("mxp", N, K)), blocks(M, K, ("mxp-x", M, K))
    Y = torch.full((M * N + 64,), 7.0, device=DEV)
    bqm.qmm_mxfp4(packed(w), packed(x), Y, M, N, K)
    got = host(Y)
    assert (got[M * N:] == 7.0).all()
    close(got[:M * N].reshape(M, N), *_mxref.product(_mxref.dequantize(w), _mxref.dequantize(x)), K, "qmm")


@pytest.mark.parametrize("M,N,K", [(7, 100, 768), (200, 300, 768)])
def test_qmm_exact_and_nan(M, N, K):
    say("qmm exact", M, N, K)
    w, x = blocks(N, K, ("mxpe",), 126, 128), blocks(M, K, ("mxpe-x",), 126, 128)
    Y = torch.empty((M, N), device=DEV)
    bqm.qmm_mxfp4(packed(w), packed(x), Y, M, N, K)
    want = _mxref.dequantize(x) @ _mxref.dequantize(w).T  # multiples of 1/16 far below 2^20: exact in fp32
    assert np.array_equal(host(Y), want.astype(np.float32))
    w[N - 1, 1, 0] = x[2, 0, 0] = 255
    bqm.qmm_mxfp4(packed(w), packed(x), Y, M, N, K)
    nan = np.zeros((M, N), bool)
    nan[2], nan[:, N - 1] = True, True
    assert np.array_equal(np.isnan(host(Y)), nan)


def test_qmm_extreme_scales_and_empty():
    say("qmm extreme scales")
    M, N, K = 20, 40, 256
    w, x = blocks(N, K, ("mxps",), 0, 4), blocks(M, K, ("mxps-x",), 250, 254)
    Y = torch.empty((M, N), device=DEV)
    bqm.qmm_mxfp4(packed(w), packed(x), Y, M, N, K)
    close(host(Y), *_mxref.product(_mxref.dequantize(w), _mxref.dequantize(x)), K, "qmm scales")
    bqm.qmm_mxfp4(None, None, Y, M, N, 0)
    assert (host(Y) == 0).all()


# ---- expert-indexed product ----

@pytest.mark.parametrize("per_slot", [False, True])
@pytest.mark.parametrize("T,E,top_k,N,K", [(1, 8, 2, 33, 128), (1, 128, 8, 64, 544), (3, 5, 3, 200, 96), (17, 6, 2, 48, 1024),
                                           (40, 3, 2, 130, 288), (150, 4, 3, 100, 160), (600, 7, 1, 40, 64), (9, 300, 8, 17, 32),
                                           (20, 4, 2, 70, 160), (256, 128, 8, 3300, 32), (1600, 128, 8, 1100, 32)])
def test_qmm_id(T, E, top_k, N, K, per_slot):
    say("qmm_id_mxfp4", T, E, top_k, N, K, per_slot)
    w = blocks(E * N, K, ("mxi", E, N, K))
    ids = gen.router_ids(T, E, top_k, ("mxi-ids", T, E))
    ids.reshape(-1)[:: 7] = -1                          # padding slots
    if T > 2:
        ids[1, 0], ids[2, :] = E, -5                     # out of range, and a token without an expert
        ids[T - 1, :] = ids[T - 1, 0]                    # the same expert for every slot of a token
    rows = T * top_k if per_slot else T
    xt, xs = (top_k, 1) if per_slot else (1, 0)
    x = blocks(rows, K, ("mxi-x", rows, K))
    Y = torch.full((T * top_k * N + 64,), 7.0, device=DEV)
    bqm.qmm_id_mxfp4(packed(w), E, N, K, torch.from_numpy(ids).to(DEV), T, top_k, packed(x), rows, xt, xs, Y)
    got = host(Y)
    assert (got[T * top_k * N:] == 7.0).all()
    want, S = _mxref.product_id(_mxref.dequantize(w), E, N, _mxref.dequantize(x), ids, xt, xs)
    close(got[:T * top_k * N].reshape(T, top_k, N), want, S, K, "qmm_id")


def test_qmm_id_edges():
    say("qmm_id edges")
    ids = torch.tensor([[0, -1], [3, 1]], dtype=torch.int32, device=DEV)
    Y = torch.full((2, 2, 5), 7.0, device=DEV)
    bqm.qmm_id_mxfp4(None, 0, 5, 64, ids, 2, 2, None, 2, 1, 0, Y)  # no experts: every id is out of range or padding
    got = host(Y)
    assert np.isnan(got[0, 0]).all() and (got[0, 1] == 0).all() and np.isnan(got[1]).all()
    bqm.qmm_id_mxfp4(None, 4, 5, 0, ids, 2, 2, None, 2, 1, 0, Y)   # K = 0: empty sums
    assert (host(Y) == 0).all()


def test_qmm_id_long_prompt():
    """Many slots of few experts, and the largest token count."""
    for T, E, top_k, N, K in ((16384, 3, 2, 16, 32), (2000, 2, 4, 300, 64)):
        say("qmm_id long", T, E, top_k, N, K)
        w, x = blocks(E * N, K, ("mxl", E)), blocks(T, K, ("mxl-x", T))
        g = np.random.default_rng(5)
        ids = g.integers(-1, E, (T, top_k), dtype=np.int32)
        Y = torch.empty((T, top_k, N), device=DEV)
        bqm.qmm_id_mxfp4(packed(w), E, N, K, torch.from_numpy(ids).to(DEV), T, top_k, packed(x), T, 1, 0, Y)
        W, X = _mxref.dequantize(w).reshape(E, N, K), _mxref.dequantize(x)
        every = np.einsum("enk,tk->ten", W, X)
        size = np.einsum("enk,tk->ten", np.abs(W), np.abs(X))
        at = np.maximum(ids, 0)[..., None]
        pad = (ids < 0)[..., None]
        close(host(Y), np.where(pad, 0, np.take_along_axis(every, at, 1)), np.where(pad, 0, np.take_along_axis(size, at, 1)), K, "long")


def test_offsets_past_32_bits():
    """Codes of more than 4 GiB and rows of more than 2^32 values: every call, checked at rows on both sides."""
    N, K, E = 1050003, 8192, 3
    say("large offsets", N, K)
    g = torch.Generator(DEV).manual_seed(11)
    b = torch.randint(0, 256, (N, K // 32, 17), dtype=torch.uint8, device=DEV, generator=g)
    b[..., 0] = torch.randint(118, 133, (N, K // 32), dtype=torch.uint8, device=DEV, generator=g)
    w = room(N, K)
    bqm.bqm_repack("mxfp4", b, w, N, K)
    assert torch.equal(unpacked(w, N, K), b)
    rows = torch.tensor([0, 15, 16, N // 3, N // 3 - 1, N // 2, 2 * (N // 3), (1 << 20) - 1, 1 << 20, N - 17, N - 1], device=DEV)
    raw = host(b[rows])
    del b
    W = _mxref.dequantize(raw)
    for M in (1, 8):
        X, Y = gen.normal((M, K), ("mxo", M)), torch.empty((M, N), device=DEV)
        bqm.qmv_mxfp4(w, X.to(DEV), Y, M, N, K)
        close(host(Y[:, rows]), *_mxref.product(W, X.numpy().astype(np.float64)), K, "qmv")
    for M in (3, 300):
        x, Y = blocks(M, K, ("mxo-x", M)), torch.empty((M, N), device=DEV)
        bqm.qmm_mxfp4(w, packed(x), Y, M, N, K)
        close(host(Y[:, rows]), *_mxref.product(W, _mxref.dequantize(x)), K, "qmm")
        ids = torch.arange(M, dtype=torch.int32, device=DEV).remainder(E)[:, None].contiguous()
        Y = torch.empty((M, N // E), device=DEV)
        bqm.qmm_id_mxfp4(w, E, N // E, K, ids, M, 1, packed(x), M, 1, 0, Y)
        want, S = _mxref.product(W, _mxref.dequantize(x))
        for k, row in enumerate(rows.tolist()):
            e, n = divmod(row, N // E)
            mine = slice(e, M, E)
            close(host(Y[mine, n]), want[mine, k], S[mine, k], K, "qmm_id")
    y = torch.empty((N, K), dtype=torch.bfloat16, device=DEV)
    bqm.bqm_dequantize_mxfp4(w, y, K, N, K)
    assert np.array_equal(host(y[rows].float()).astype(np.float64), W)  # codes times powers of two are exact in bf16
    bqm.bqm_quantize_mxfp4(y, K, w, N, K)
    assert np.array_equal(host(unpacked(w, N, K)[rows]), _mxref.quantize(W))


# ---- together, and in graphs ----

def layer(T, E, top_k, H, F, key):
    """A mixture-of-experts feed-forward layer as a program runs it: router logits by the decode product or the prefill
    one, routing, gate and up, SwiGLU, down, the weighted sum of each token's experts."""
    b = {n: blocks(r, k, key + (n,), 118, 122) for n, r, k in (("r", E, H), ("g", E * F, H), ("u", E * F, H), ("d", E * H, F))}
    w = {n: packed(v) for n, v in b.items()}
    x = gen.normal((T, H), key + ("x",), device=DEV)
    bias = gen.normal((E,), key + ("b",), std=0.05, device=DEV)
    s = dict(x=x, logits=torch.empty((T, E), device=DEV), ids=torch.empty((T, top_k), dtype=torch.int32, device=DEV),
             rw=torch.empty((T, top_k), device=DEV), xp=room(T, H), hp=room(T * top_k, F),
             g=torch.empty((T, top_k, F), device=DEV), u=torch.empty((T, top_k, F), device=DEV),
             d=torch.empty((T, top_k, H), device=DEV), y=torch.empty((T, H), device=DEV))

    def run():
        bqm.bqm_quantize_mxfp4(x, H, s["xp"], T, H)
        if T <= 8:
            bqm.qmv_mxfp4(w["r"], x, s["logits"], T, E, H)
        else:
            bqm.qmm_mxfp4(w["r"], s["xp"], s["logits"], T, E, H)
        bqm.bqm_route("sigmoid", s["logits"], E, bias, T, E, 2, 1, 2, top_k, True, 1.5, s["ids"], s["rw"])
        bqm.qmm_id_mxfp4(w["g"], E, F, H, s["ids"], T, top_k, s["xp"], T, 1, 0, s["g"])
        bqm.qmm_id_mxfp4(w["u"], E, F, H, s["ids"], T, top_k, s["xp"], T, 1, 0, s["u"])
        h = torch.nn.functional.silu(s["g"]) * s["u"]
        bqm.bqm_quantize_mxfp4(h, F, s["hp"], T * top_k, F)
        bqm.qmm_id_mxfp4(w["d"], E, H, F, s["ids"], T, top_k, s["hp"], T * top_k, top_k, 1, s["d"])
        s["y"].copy_((s["d"] * s["rw"][..., None]).sum(1))

    return b, s, bias, run


@pytest.mark.parametrize("T", [1, 7, 50])
def test_moe_layer(T):
    say("moe layer", T)
    E, top_k, H, F = 16, 3, 256, 96
    b, s, bias, run = layer(T, E, top_k, H, F, ("mxlayer",))
    run()
    # each stage against its plain form on the stage's own inputs
    X, W = host(s["x"]).astype(np.float64), {n: _mxref.dequantize(v) for n, v in b.items()}
    Xq = _mxref.dequantize(_mxref.quantize(X))
    close(host(s["logits"]), *_mxref.product(W["r"], X if T <= 8 else Xq), H, "logits")
    ids, rw = _mxref.route(host(s["logits"]), host(bias), "sigmoid", 2, 1, 2, top_k, True, 1.5)
    assert np.array_equal(host(s["ids"]), ids) and np.abs(host(s["rw"]) - rw).max() <= 2.0 ** -23 * 1.5
    for n in "gu":
        close(host(s[n]), *_mxref.product_id(W[n], E, F, Xq, ids, 1, 0), H, n)
    h = host(torch.nn.functional.silu(s["g"]) * s["u"]).reshape(T * top_k, F)
    Hq = _mxref.dequantize(_mxref.quantize(h))
    close(host(s["d"]), *_mxref.product_id(W["d"], E, H, Hq, ids, top_k, 1), F, "down")
    y = (host(s["d"]).astype(np.float64) * host(s["rw"])[..., None]).sum(1)
    size = np.abs(host(s["d"]).astype(np.float64) * host(s["rw"])[..., None]).sum(1)
    assert (np.abs(host(s["y"]) - y) <= (top_k + 1) * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("T", [2, 40])
def test_graph_of_the_layer(T):
    say("graph: moe layer in MXFP4", T)
    _, s, _, run = layer(T, 16, 3, 256, 96, ("mxgraph",))
    replays_match_eager(run, [s["logits"], s["rw"], s["g"], s["u"], s["d"], s["y"]])


def test_graph_of_the_dense_products():
    say("graph: dense products in MXFP4")
    M, N, K = 300, 520, 1056
    w = packed(blocks(N, K, ("mxgd",)))
    x = gen.normal((M, K), ("mxgd-x",), device=DEV).to(torch.bfloat16)
    xp, back = room(M, K), torch.empty((M, K), device=DEV)
    Y, V = torch.empty((M, N), device=DEV), torch.empty((8, N), device=DEV)
    xv = gen.normal((8, K), ("mxgd-v",), device=DEV)

    def run():
        bqm.bqm_quantize_mxfp4(x, K, xp, M, K)
        bqm.bqm_dequantize_mxfp4(xp, back, K, M, K)
        bqm.qmm_mxfp4(w, xp, Y, M, N, K)
        bqm.qmv_mxfp4(w, xv, V, 8, N, K)

    replays_match_eager(run, [back, Y, V])

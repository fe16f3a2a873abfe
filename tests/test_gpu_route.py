"""Routing to experts on the GPU against the plain 64-bit form: ids equal, weights to the last bit or two of fp32."""
import numpy as np
import pytest
import torch

import gen
import oracle
from block_quantized_matrix_amd import bqm
from tests import _mxref
from tests._gpu import DEV, check_close, host, packed, say, weights
from tests.test_gpu_graphs import replays_match_eager

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def route(logits, bias, score, n_group, topk_group, group_top, top_k, renorm, scale):
    T, E = logits.shape
    ids = torch.full((T * top_k + 32,), 77, dtype=torch.int32, device=DEV)
    w = torch.full((T * top_k + 32,), 7.0, device=DEV)
    bqm.bqm_route(score, logits, logits.stride(0), bias, T, E, n_group, topk_group, group_top, top_k, renorm, scale, ids, w)
    ids, w = host(ids), host(w)
    assert (ids[T * top_k:] == 77).all() and (w[T * top_k:] == 7.0).all()
    return ids[:T * top_k].reshape(T, top_k), w[:T * top_k].reshape(T, top_k)


def check(logits, bias, *a):
    ids, w = route(logits, bias, *a)
    want_ids, want = _mxref.route(host(logits.float()), None if bias is None else host(bias), *a)
    assert np.array_equal(ids, want_ids)
    # 64-bit arithmetic on both sides, rounded once to fp32: half a step (2^-24), and as much again for the 64 bits'
    # own errors next to a rounding border; below 2^-126 a step is 2^-149
    assert np.array_equal(np.isnan(w), np.isnan(want))
    d = np.abs(np.nan_to_num(w.astype(np.float64)) - np.nan_to_num(want))
    assert (d <= 2.0 ** -23 * np.abs(np.nan_to_num(want)) + 2.0 ** -149).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,E,top_k", [(1, 1, 1), (1, 128, 8), (3, 7, 7), (5, 60, 4), (33, 64, 6), (200, 128, 8), (65, 256, 8), (9, 1000, 32),
                                       (2, 4096, 32), (17, 96, 2), (130, 16, 16), (4, 5, 9)])
def test_route(T, E, top_k, dtype, score):
    say("route", T, E, top_k, dtype, score)
    l = (gen.normal((T, E), ("route", T, E), device=DEV) * 2).to(TYPES[dtype])
    bias = gen.normal((E,), ("route-b", E), std=0.1, device=DEV)
    for b in (None, bias):
        for renorm, scale in ((True, 1.0), (False, 2.5)):
            check(l, b, score, 1, 1, 1, top_k, renorm, scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,top_k", [(256, 8, 4, 8), (64, 8, 3, 6), (60, 3, 1, 8), (160, 16, 16, 4), (128, 64, 5, 9),
                                                        (4096, 64, 7, 32), (30, 5, 2, 12), (9, 9, 3, 4)])
def test_groups(E, n_group, topk_group, top_k, score):
    say("route groups", E, n_group, topk_group, top_k, score)
    for dtype in (torch.float32, torch.bfloat16):
        l = (gen.normal((37, E), ("route-g", E), device=DEV) * 1.5).to(dtype)
        bias = gen.normal((E,), ("route-gb", E), std=0.05, device=DEV)
        for b in (None, bias):
            for group_top in (1, 2):
                if group_top <= E // n_group:
                    check(l, b, score, n_group, topk_group, group_top, top_k, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,top_k", [(256, 8, 3, 8), (60, 3, 1, 6)])
@pytest.mark.parametrize("T", [5, 1101])
def test_group_sums_beyond_fp32(T, E, n_group, topk_group, top_k, score):
    """Biases whose sums pass the range of fp32, or lie on its last step, keep the order that 64 bits give them."""
    say("route group sums", T, E, n_group, topk_group, top_k, score)
    l = gen.normal((T, E), ("route-o", T, E), device=DEV)
    g = torch.arange(n_group, dtype=torch.float64)
    for base, step in ((2.0e38, 2.0e35), (1.0, 2.0 ** -22)):
        bias = torch.zeros(n_group, E // n_group, dtype=torch.float64)
        bias[:, 0], bias[:, 3] = base + step * g, base
        check(l, bias.reshape(-1).float().to(DEV), score, n_group, topk_group, 2, top_k, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_index(score):
    say("route ties", score)
    l = torch.from_numpy(np.random.default_rng(2).integers(-2, 3, (60, 96)).astype(np.float32)).to(DEV)
    bias = torch.from_numpy(np.random.default_rng(3).integers(0, 2, 96).astype(np.float32) / 4).to(DEV)
    flat = torch.zeros_like(l)
    for x in (l, flat):
        for g, kg, gt in ((1, 1, 1), (8, 3, 1), (8, 3, 2)):
            check(x, None, score, g, kg, gt, 8, True, 1.0)
            check(flat if x is flat else (x > 0).float(), bias, score, g, kg, gt, 8, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_neighbours_in_the_last_bit(score):
    """Logits a single step apart, and scores whose order only 64 bits show."""
    say("route neighbours", score)
    g = np.random.default_rng(4)
    l = (np.float32(1) + g.integers(0, 200, (64, 128)).astype(np.float32) * np.float32(2.0 ** -23))
    check(torch.from_numpy(l).to(DEV), None, score, 1, 1, 1, 8, True, 1.0)
    bias = torch.from_numpy((g.integers(0, 50, 128) * 2.0 ** -30).astype(np.float32)).to(DEV)
    check(torch.from_numpy(l).to(DEV), bias, score, 1, 1, 1, 8, True, 1.0)
    check(torch.from_numpy(l).to(DEV), bias, score, 8, 3, 2, 8, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks_and_specials(score):
    say("route masks", score)
    inf, nan = float("inf"), float("nan")
    l = gen.normal((12, 40), ("route-m",), device=DEV)
    l[0, :] = -inf                      # no expert left
    l[1, 3:] = -inf                     # fewer than top_k
    l[2, ::2] = -inf
    l[3, 7] = nan
    l[4, 9] = inf
    least, most = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    l[5, :] = least                       # a mask of the lowest value is a number: all alike
    l[6, 1:] = least
    l[7, :] = most
    l[8, :] = -1000.0                   # sigmoid scores that are 0 even in 64 bits
    l[9, 10:20] = -inf                  # one whole group gone
    l[10, 5], l[10, 6] = inf, -inf
    bias = gen.normal((40,), ("route-mb",), std=0.1, device=DEV)
    low = bias.clone()
    low[4] = -inf
    bad = bias.clone()
    bad[11] = nan
    for b in (None, bias, low, bad):
        for g, kg, gt in ((1, 1, 1), (4, 2, 1), (4, 2, 2)):
            for renorm in (True, False):
                check(l, b, score, g, kg, gt, 6, renorm, 1.0)
    for dtype in (torch.float16, torch.bfloat16):
        x = l.clone()
        x[5, :], x[6, 1:], x[7, :] = torch.finfo(dtype).min, torch.finfo(dtype).min, torch.finfo(dtype).max
        check(x.to(dtype), bias, score, 4, 2, 2, 6, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E,n_group,topk_group,top_k", [(60, 1, 1, 8), (64, 4, 2, 6), (128, 1, 1, 8), (96, 3, 2, 30), (250, 5, 2, 8),
                                                        (256, 8, 4, 8), (256, 64, 9, 32)])
def test_long_prompts(E, n_group, topk_group, top_k, dtype, score):
    """Prompts take fewer lanes a token and select by 32-bit keys first: random logits, ties, steps in the last bit, values
    that only 64 bits tell apart, masks and NaN, all in one batch."""
    say("route long", E, n_group, topk_group, top_k, dtype, score)
    T, g, t = 1101, np.random.default_rng(E), TYPES[dtype]
    l = gen.normal((T, E), ("route-long", E), device=DEV) * 1.5
    l[300:400] = torch.from_numpy(g.integers(-2, 3, (100, E)).astype(np.float32)).to(DEV)          # ties
    l[400:500] = torch.from_numpy(1 + g.integers(0, 200, (100, E)) * 2.0 ** -23).float().to(DEV)   # neighbours
    l[500:520] = 0
    l[520:540, ::3] = float("-inf")
    l[540:550, 2:] = float("-inf")
    l[550] = float("-inf")
    l[551, 5], l[552, 7], l[553, 1] = float("nan"), float("inf"), torch.finfo(torch.float32).min
    l = l.to(t)
    random = gen.normal((E,), ("route-long-b", E), std=0.05, device=DEV)
    steps = torch.from_numpy((g.integers(0, 50, E) * 2.0 ** -30).astype(np.float32)).to(DEV)
    wide = random.clone()
    wide[::7] *= 1e6
    for bias in (None, random, torch.zeros_like(random), steps, wide):
        for group_top in (1, 2) if n_group > 1 else (1,):
            check(l, bias, score, n_group, topk_group, group_top, top_k, True, 1.0)
    check(l, random, score, n_group, topk_group, 1, min(top_k, 3), False, 2.5)


def test_strides_and_empty():
    say("route strides")
    for dtype in TYPES.values():
        wide = (gen.normal((50, 131), ("route-s",), device=DEV) * 2).to(dtype)
        check(wide[:, :97], None, "softmax", 1, 1, 1, 5, True, 1.0)
    ids, w = route(torch.empty((3, 0), device=DEV), None, "softmax", 1, 1, 1, 4, True, 1.0)
    assert (ids == -1).all() and (w == 0).all()


def test_many_tokens():
    say("route many tokens")
    l = gen.normal((70000, 24), ("route-many",), device=DEV)
    ids, w = route(l, None, "softmax", 1, 1, 1, 2, True, 1.0)
    x = host(l).astype(np.float64)
    order = np.argsort(-x, axis=1, kind="stable")[:, :2]
    assert np.array_equal(ids, order)
    z = np.exp(np.take_along_axis(x, order, 1))
    assert np.abs(w - z / z.sum(1, keepdims=True)).max() <= 2.0 ** -23


def test_graph():
    say("graph: route")
    l = gen.normal((300, 64), ("route-graph",), device=DEV)
    bias = gen.normal((64,), ("route-graph-b",), std=0.05, device=DEV)
    ids, w = torch.empty((300, 6), dtype=torch.int32, device=DEV), torch.empty((300, 6), device=DEV)
    kept = torch.empty((300, 6), device=DEV)

    def run():
        bqm.bqm_route("sigmoid", l, 64, bias, 300, 64, 8, 3, 2, 6, True, 1.0, ids, w)
        kept.copy_(ids)

    replays_match_eager(run, [w, kept])


def test_router_in_front_of_the_q4_0_experts():
    """Ids and weights as the router leaves them go straight into the Q4_0 experts' products, a masked token among them."""
    say("route + qmv_id_gate_up + qmv_id_sum")
    oracle.build(force=False)
    T, E, top_k, H, F = 5, 12, 3, 512, 128
    l = gen.normal((T, E), ("route-moe",), device=DEV)
    l[2, 2:] = float("-inf")
    ids, rw = torch.empty((T, top_k), dtype=torch.int32, device=DEV), torch.empty((T, top_k), device=DEV)
    wg, wu = weights("q4_0", E * F, H, ("route-moe", 0)), weights("q4_0", E * F, H, ("route-moe", 1))
    wd = weights("q4_0", E * H, F, ("route-moe", 2))
    x = gen.normal((T, H), ("route-moe-x",), device=DEV)
    h, ys, y = torch.empty((T, top_k, F), device=DEV), torch.empty((T, top_k, H), device=DEV), torch.empty((T, H), device=DEV)
    pg, pu, pd = packed("q4_0", wg, E * F, H), packed("q4_0", wu, E * F, H), packed("q4_0", wd, E * H, F)
    bqm.bqm_route("softmax", l, E, None, T, E, 1, 1, 1, top_k, True, 1.0, ids, rw)
    bqm.qmv_id_gate_up("q4_0", pg, pu, E, F, H, ids, T, top_k, x, H, 0, h)
    bqm.qmv_id_sum("q4_0", pd, E, H, F, ids, rw, T, top_k, h, top_k * F, F, ys, y)
    want_ids, want = _mxref.route(host(l), None, "softmax", 1, 1, 1, top_k, True, 1.0)
    assert np.array_equal(host(ids), want_ids) and want_ids[2, 2] == -1
    yr, S = oracle.qmv_id_sum("q4_0", host(wd), E, H, F, want_ids, want.astype(np.float32), host(h).reshape(-1), top_k * F, F)
    check_close(host(y), yr, S, "moe")

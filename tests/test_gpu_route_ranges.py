"""The router at the ends of its numbers' ranges, against the plain 64-bit form: sums of two biases below fp32's range,
sigmoid scores at the end of 64 bits, and groups of more than 256 experts."""
import numpy as np
import pytest
import torch

import gen
from tests import _mxref
from tests._gpu import DEV, host, say
from tests.test_gpu_route import TYPES, route

pytestmark = pytest.mark.gpu


def check(logits, bias, *a):
    """Some forty of the tokens, the last among them, against the plain form: ids equal, weights within half a step of
    fp32 (2^-24) and as much again for the 64 bits' own errors next to a rounding border."""
    ids, w = route(logits, bias, *a)
    T = logits.shape[0]
    some = np.unique(np.r_[0:min(T, 12), np.linspace(0, T - 1, 30).astype(int)])
    want_ids, want = _mxref.route(host(logits.float())[some], None if bias is None else host(bias), *a)
    assert np.array_equal(ids[some], want_ids)
    assert np.array_equal(np.isnan(w[some]), np.isnan(want))
    d = np.abs(np.nan_to_num(w[some].astype(np.float64)) - np.nan_to_num(want))
    assert (d <= 2.0 ** -23 * np.abs(np.nan_to_num(want)) + 2.0 ** -149).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,top_k", [(256, 8, 3, 8), (64, 4, 2, 6), (60, 3, 1, 6), (128, 64, 5, 9)])
@pytest.mark.parametrize("T", [5, 1101])
def test_group_sums_below_fp32(T, E, n_group, topk_group, top_k, score):
    """Two finite values whose sum passes the lowest fp32: such groups keep the order of their real sums, and stay above a
    group that has no expert at all."""
    say("route group sums below", T, E, n_group, topk_group, top_k, score)
    size, least = E // n_group, torch.finfo(torch.float32).min
    l = gen.normal((T, E), ("route-below", T, E), device=DEV)
    empty = l.clone()
    empty[:, :size] = float("-inf")   # the first group has no expert
    rising = torch.linspace(-3.3e38, -2.0e38, n_group, dtype=torch.float64)  # the better ones last
    masked = torch.full((n_group,), least, dtype=torch.float64)
    masked[-1] = 0.0
    some = rising.clone()
    some[::2] = 0.0
    mixed = rising.clone()
    mixed[1] = 3.0e38
    for x in (l, empty):
        for bias in (rising, masked, some, mixed, torch.full((n_group,), least, dtype=torch.float64)):
            for apart in (0.0, 0.1):  # a group's experts alike, or well apart
                b = bias.repeat_interleave(size) * (1 - apart * torch.arange(E).remainder(size) / size)
                b = b.float().to(DEV)
                check(x, b, score, n_group, topk_group, 2, top_k, True, 1.0)
            b[::size] = 0.0   # one usable expert in every group
            check(x, b, score, n_group, topk_group, 2, top_k, True, 1.0)


def test_masked_groups_by_hand():
    """Group 0 without an expert, groups 1 and 2 masked by the lowest number, two groups to keep: 3 and 1."""
    say("route masked groups")
    for T in (3, 1100):
        l = torch.zeros((T, 64), device=DEV)
        l[:, :16] = float("-inf")
        bias = torch.zeros(64, device=DEV)
        bias[16:48] = torch.finfo(torch.float32).min
        ids, w = route(l, bias, "sigmoid", 4, 2, 2, 18, True, 1.0)
        assert (ids == np.r_[48:64, 16:18]).all() and (w == np.float32(1 / 18)).all()


@pytest.mark.parametrize("T", [4, 1030])
@pytest.mark.parametrize("E", [40, 200, 300])
def test_sigmoid_at_the_end_of_64_bits(E, T):
    """Scores down to the reciprocal of the largest 64-bit number, 709.78 below zero, where they are 0 from there on."""
    say("route sigmoid end", E, T)
    l = torch.linspace(-709.9, -708.2, E, device=DEV).repeat(T, 1)
    l[1::2] = l[1::2].flip(1)
    zero, bias = torch.zeros(E, device=DEV), torch.zeros(E, device=DEV)
    l[2, 6:], bias[:3] = -800.0, -1.0  # scores of 0 beside six small ones
    l[2, :6] = torch.linspace(-709.78, -708.2, 6)
    for b in (None, zero, bias):
        for renorm in (True, False):
            check(l, b, "sigmoid", 1, 1, 1, 8, renorm, 1.0)
    check(l, zero, "sigmoid", 4, 2, 2, 8, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,E,n_group,topk_group,top_k", [(37, 257, 1, 1, 8), (40, 264, 8, 3, 8), (1030, 384, 6, 2, 5), (9, 510, 3, 2, 32),
                                                          (70, 512, 16, 4, 8), (5, 513, 27, 9, 10)])
def test_more_than_256_experts(T, E, n_group, topk_group, top_k, dtype, score):
    say("route many experts", T, E, n_group, topk_group, top_k, dtype, score)
    g = np.random.default_rng(E)
    l = gen.normal((T, E), ("route-256", T, E), device=DEV) * 1.5
    l[1] = torch.from_numpy(g.integers(-2, 3, E).astype(np.float32)).to(DEV)
    l[2], l[3, ::3], l[4, :] = 0.0, float("-inf"), float("-inf")
    l = l.to(TYPES[dtype])
    random = gen.normal((E,), ("route-256-b", E), std=0.05, device=DEV)
    out = random.clone()
    out[5::7] = float("-inf")
    for bias in (None, random, out):
        for group_top in (1, 2) if n_group > 1 else (1,):
            check(l, bias, score, n_group, topk_group, group_top, top_k, True, 1.0)

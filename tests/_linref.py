"""Plain NumPy forms, in 64 bits, of the calls on float rows (include/bqm.h defines them), and how far the kernels may be
from them."""
import math

import numpy as np
import torch

import gen
from tests import _mxref

FMTS = ("q4_0", "q8_0", "mxfp4")
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
BLOCK = {"q4_0": 18, "q8_0": 34, "mxfp4": 17}


def blocks(fmt, rows, K, key, top=1.0):
    """Random interchange blocks [rows, K/32, bytes]: every code, scales of both signs (MXFP4: powers of two) around
    top / 100."""
    g = np.random.default_rng(gen.seed_of("lin", fmt, rows, K, *key))
    b = g.integers(0, 256, (rows, K // 32, BLOCK[fmt]), dtype=np.uint8)
    if fmt == "mxfp4":
        b[..., 0] = g.integers(117, 123, (rows, K // 32))
    else:
        d = (g.normal(size=(rows, K // 32)) * top / 100).astype(np.float16)
        b[..., :2] = d[..., None].view(np.uint8)
        if fmt == "q8_0":
            body = b[..., 2:]
            body[body == 128] = 0
    return b


def dequantize(fmt, b):
    """Interchange bytes [rows, nb, bytes] -> fp64 [rows, 32 nb]."""
    if fmt == "mxfp4":
        return _mxref.dequantize(b)
    d = np.ascontiguousarray(b[..., :2]).view(np.float16).astype(np.float64)
    body = np.ascontiguousarray(b[..., 2:])
    codes = body.view(np.int8).astype(np.float64) if fmt == "q8_0" else \
        np.concatenate([body & 15, body >> 4], -1).astype(np.float64) - 8
    return (codes * d).reshape(b.shape[0], -1)


def act(name, z):
    with np.errstate(all="ignore"):
        if name == "relu":
            return np.where(z < 0, 0.0, z)
        if name == "silu":
            return z / (1 + np.exp(-z))
        if name == "gelu":
            return 0.5 * z * torch.special.erfc(torch.from_numpy(-z * math.sqrt(0.5))).numpy()
        if name == "gelu_tanh":
            return z / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def linear(W, X, bias=None, activation="none", mul=None, res=None):
    """(y, |z| scale): y in fp64, and S = sum |w x| + |bias|, which the error of z goes by."""
    with np.errstate(all="ignore"):
        z, S = X @ W.T, np.abs(X) @ np.abs(W).T
        if bias is not None:
            z, S = z + bias, S + np.abs(bias)
        y = act(activation, z)
        if mul is not None:
            y = y * mul
        if res is not None:
            y = y + res
    return y, S


def tolerance(y, S, K, out, mul=None, res=None):
    """Bound of |got - y|.  The sum: fp32 sums of exact products, one result added per block, in at most a few shares
    (_mxref.tolerance); fp32 rows go as three parts, whose magnitudes add up to less than 1 + 2^-6 of theirs: one part in
    eight more.  No activation's slope is above 1.13.  Its own error, of its value (at most |z| <= S): exp and erfc to a
    few steps of 2^-23, the argument of exp in gelu_tanh is rounded five times and that of erfc twice, which counts
    against the value by |u| e^-|u| < 0.37 and t^2 e^-t^2 / sqrt(pi) < 0.21 of |z|: 16 steps of 2^-23 in all.  The product
    with mul and the sum with the residual round once each, relative to what they give; and half a step of out's type,
    or of its smallest numbers.  Below 2^-126 fp32 has only the multiples of 2^-149, whatever the relative error: K
    terms are added, each sum off by half of that at most, which mul scales."""
    m = 1.0 if mul is None else np.abs(mul)
    err = (1.13 * 1.125 * _mxref.tolerance(K) + 16 * 2.0 ** -23) * S * m + K * 2.0 ** -150 * m
    mag = np.abs(y) + (0 if res is None else np.abs(res))
    f = torch.finfo(out)
    err = err + 2.0 ** -23 * mag
    return err + f.eps / 2 * (np.abs(y) + err) + f.tiny * f.eps


def close(got, y, tol, what):
    """NaN and infinities in their places, the rest within tol."""
    got = np.asarray(got, np.float64)
    odd = ~np.isfinite(y)
    assert np.array_equal(got[odd], y[odd], equal_nan=True), f"{what}: infinities or NaN in other places"
    with np.errstate(all="ignore"):
        err = np.where(odd, 0, np.abs(got - y))
    bad = ~(err <= np.where(odd, 0, tol))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outputs off, first at {np.argwhere(bad)[0].tolist()}, " \
                          f"worst {np.nanmax(np.where(bad, err / np.maximum(tol, 1e-300), 0))} of the tolerance"

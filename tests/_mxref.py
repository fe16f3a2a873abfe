"""Plain NumPy forms, in 64 bits, of the MXFP4 calls and the router (include/bqm.h defines them)."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def quantize(x):
    """Float rows [rows, K] -> interchange bytes [rows, K/32, 17], value by value from the definition."""
    v = np.asarray(x, np.float64).reshape(x.shape[0], -1, 32)
    out = np.zeros(v.shape[:2] + (17,), np.uint8)
    fine = np.isfinite(v).all(-1)
    v = np.where(fine[..., None], v, 0.0)
    top = np.abs(v).max(-1)
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1))[1] - 1 - 2, -127)
    e = np.maximum(e, -127)
    a = np.abs(v) * np.ldexp(1.0, -e)[..., None]
    code = np.zeros(v.shape, np.int64)
    for c in range(8):  # nearest of the grid; of two as near, the even code
        d, best = np.abs(a - GRID[c]), np.abs(a - GRID[code])
        code = np.where((d < best) | ((d == best) & (c % 2 == 0)), c, code)
    code = code + 8 * np.signbit(v)
    out[..., 0] = np.where(fine, e + 127, 255)
    code = np.where(fine[..., None], code, 0)
    out[..., 1:] = code[..., :16] | code[..., 16:] << 4
    return out


def dequantize(blocks):
    """Interchange bytes [rows, nb, 17] -> fp64 [rows, 32 nb]."""
    b = np.asarray(blocks, np.uint8)
    codes = np.concatenate([b[..., 1:] & 15, b[..., 1:] >> 4], -1)
    e = b[..., 0].astype(np.int64)
    scale = np.where(e == 255, np.nan, np.ldexp(1.0, e - 127))
    return (np.where(codes >= 8, -1.0, 1.0) * GRID[codes & 7] * scale[..., None]).reshape(b.shape[0], -1)


def product(W, X):
    """Y = X W^T in fp64, and the sum of the terms' magnitudes."""
    return X @ W.T, np.abs(X) @ np.abs(W).T


def product_id(W, E, N, X, ids, x_tok_rows, x_slot_rows):
    T, top_k = ids.shape
    Y, S = np.zeros((T, top_k, N)), np.zeros((T, top_k, N))
    for t in range(T):
        for s in range(top_k):
            e = ids[t, s]
            if e >= E:
                Y[t, s] = np.nan
            elif e >= 0:
                r = t * x_tok_rows + s * x_slot_rows
                Y[t, s], S[t, s] = (v[0] for v in product(W[e * N:(e + 1) * N], X[r:r + 1]))
    return Y, S


def tolerance(K):
    """Bound of |y - y64| / sum |w x| for products of K terms whose products are exact: fp32 sums that add one result per
    block of 32 (K / 32 of them, an error of a step of 2^-23 each, truncation included), at most 32 terms inside a
    block and 8 sums at the end."""
    return (K / 32 + 40) * 2.0 ** -23


def route(logits, bias, score, n_group, topk_group, group_top, top_k, renorm, scale):
    """ids int32 and weights fp64 [T, top_k], one token at a time."""
    T, E = logits.shape
    ids, weights = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    for t in range(T):
        l = np.asarray(logits[t], np.float64)
        b = None if bias is None else np.asarray(bias, np.float64)
        if np.isnan(l).any() or (b is not None and np.isnan(b).any()) or (score == "softmax" and (l == np.inf).any()):
            n = min(top_k, E)
            ids[t, :n], weights[t, :n] = np.arange(n), np.nan
            continue
        with np.errstate(all="ignore"):
            if score == "softmax":
                z = np.exp(l - l.max()) if E and l.max() > -np.inf else np.zeros(E)
                p = z / z.sum() if z.sum() > 0 else z
            else:
                p = 1 / (1 + np.exp(-l))
        out = l == -np.inf
        value = np.where(out, -np.inf, l if b is None else p + b)
        if n_group > 1:
            size = E // n_group
            v = np.where(out, -np.inf, p) if b is None and group_top == 2 else value
            gs = []
            for g in range(n_group):
                top = [u for u in sorted(v[g * size:(g + 1) * size], reverse=True)[:group_top] if u > -np.inf]
                gs.append(sum(top) if top else -np.inf)
            kept = sorted(range(n_group), key=lambda g: (-gs[g], g))[:topk_group]
            for g in range(n_group):
                if g not in kept:
                    value[g * size:(g + 1) * size] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-value[e], e)) if value[e] > -np.inf][:top_k]
        w = np.array([p[e] for e in order])
        if renorm and len(order):
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        ids[t, :len(order)], weights[t, :len(order)] = order, w * np.float64(np.float32(scale))
    return ids, weights

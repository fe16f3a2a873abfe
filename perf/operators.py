"""The router and the MXFP4 operators of block_quantized_matrix_amd, in plain torch and as the library's calls.

Six calls, five operators:

- route: expert ids and weights of a mixture-of-experts layer from its router's logits (bqm_route);
- quantize: rows of floats to MXFP4 (OCP microscaling: 32 e2m1 codes under one e8m0 scale) and back
  (bqm_quantize_mxfp4, bqm_dequantize_mxfp4);
- qmv: decode, MXFP4 weights times 1 to 8 fp32 vectors (qmv_mxfp4);
- qmm: prefill, MXFP4 weights times activations that are quantized to MXFP4 first (bqm_quantize_mxfp4, qmm_mxfp4);
- qmm_id: the same product with the matrices of the experts that a router chose (bqm_quantize_mxfp4, qmm_id_mxfp4).

Weights come as interchange blocks of 17 bytes: the e8m0 scale, then 16 bytes of which byte j holds code j in its low
nibble and code j + 16 in its high one.  A program repacks them once, when it loads its model, and keeps them so.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of a 128-expert layer with top-8 routing, at every layer of every decode step: pure latency
        dict(name="route one token", op="route", T=1, E=128, top_k=8, score="softmax", bias=False, n_group=1,
             topk_group=1, group_top=1, renorm=True, dtype="f32"),
        # a long prompt through a sigmoid router with a balancing bias and experts in groups
        dict(name="route a prompt, groups", op="route", T=16384, E=256, top_k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, renorm=True, dtype="bf16"),
        # the activations of a 16-token decode batch
        dict(name="quantize 16 tokens", op="quantize", rows=16, K=4096, dtype="f32"),
        # one projection of the 27B dense model, quantized as it is loaded
        dict(name="quantize a projection", op="quantize", rows=17408, K=5120, dtype="bf16"),
        # the smallest decode product of the benchmark
        dict(name="qmv 4096 x 4096", op="qmv", M=1, N=4096, K=4096),
        # gate and up of the 27B dense model stacked, one token
        dict(name="qmv 34816 x 5120", op="qmv", M=1, N=34816, K=5120),
        # down of the 27B dense model, a full decode batch
        dict(name="qmv 5120 x 17408, 8 tokens", op="qmv", M=8, N=5120, K=17408),
        # a short prompt at sizes that no tile divides
        dict(name="qmm ragged", op="qmm", M=33, N=1000, K=4128, dtype="f32"),
        # the 512-token prefill of the benchmark
        dict(name="qmm 512 tokens", op="qmm", M=512, N=17408, K=5120, dtype="bf16"),
        # a long prompt through the same projection
        dict(name="qmm 4096 tokens", op="qmm", M=4096, N=17408, K=5120, dtype="bf16"),
        # gate of the 128-expert layer, one token: eight experts' matrices, one row each
        dict(name="qmm_id one token", op="qmm_id", T=1, E=128, top_k=8, N=1536, K=4096, per_slot=False, dtype="f32"),
        # gate of the 128-expert layer over a 512-token prompt with a skewed router
        dict(name="qmm_id 512 tokens", op="qmm_id", T=512, E=128, top_k=8, N=1536, K=4096, per_slot=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "qmv", "qmm", "qmm_id"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 3, 4, 8])
        E = n_group * max(2, _log(rng, 8, 512) // n_group)
        T = _log(rng, 1, min(16384, 16384 * 256 // E))
        topk_group = rng.randint(1, n_group)
        return dict(op=op, T=T, E=E, top_k=rng.randint(1, min(16, E // n_group * topk_group)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, n_group=n_group,
                    topk_group=topk_group, group_top=rng.randint(1, 2), renorm=rng.random() < 0.7, dtype=dtype)
    K = 32 * _log(rng, 1, 544)
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 17408 * 5120 // K), K=K, dtype=dtype)
    if op == "qmv":
        return dict(op=op, M=rng.randint(1, 8), N=_log(rng, 16, min(65536, 17408 * 5120 // K)), K=K)
    if op == "qmm":
        return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 16, min(17408, 17408 * 5120 // K)), K=K, dtype=dtype)
    K = 32 * _log(rng, 4, 160)
    E = _log(rng, 4, 128)
    return dict(op=op, T=_log(rng, 1, 512), E=E, top_k=rng.randint(1, min(8, E)),
                N=_log(rng, 16, min(2048, 1536 * 4096 * 128 // (K * E))), K=K, per_slot=rng.random() < 0.5, dtype=dtype)


# ---- inputs ----

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _blocks(w):
    """Interchange blocks [rows, K/32, 17] of float rows, as a checkpoint holds them."""
    rows, K = w.shape
    v = w.reshape(rows, K // 32, 32)
    e = torch.frexp(v.abs().amax(-1, keepdim=True))[1].clamp_(min=-124, max=130) + 124
    q = v * torch.pow(2.0, (127 - e).to(torch.float32))
    a = q.abs()
    code = torch.zeros_like(v, dtype=torch.uint8)
    for edge in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):  # weights on an edge itself do not occur in earnest
        code += a > edge
    code += (q < 0).to(torch.uint8) * 8
    return torch.cat([e.to(torch.uint8), code[..., :16] | (code[..., 16:] << 4)], -1)


def _weights(g, rows, K):
    """Blocks of normal weights, made in pieces that keep the floats small."""
    piece = max(1, (1 << 27) // K)
    return torch.cat([_blocks(_normal(g, min(piece, rows - r), K) * 0.02) for r in range(0, rows, piece)])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] == "route":
        s["logits"] = (_normal(g, c["T"], c["E"]) * 1.5).to(DTYPES[c["dtype"]])
        s["bias"] = _normal(g, c["E"]) * 0.05 if c["bias"] else None
        s["ids"] = torch.empty((c["T"], c["top_k"]), dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty((c["T"], c["top_k"]), device=DEV)
        return s
    if c["op"] == "quantize":
        s["x"] = (_normal(g, c["rows"], c["K"]) * 0.02).to(DTYPES[c["dtype"]])
        s["y"] = torch.empty_like(s["x"])
        if own:
            s["xp"] = _room(c["rows"], c["K"])
        return s
    if c["op"] == "qmm_id":
        rows, n = c["T"] * c["top_k"] if c["per_slot"] else c["T"], c["E"] * c["N"]
        logits = _normal(g, c["T"], c["E"]) - 1.1 * torch.arange(1, c["E"] + 1, device=DEV).log()
        s["ids"] = logits.argsort(-1, descending=True)[:, :c["top_k"]].to(torch.int32).contiguous()
        s["y"] = torch.empty((c["T"], c["top_k"], c["N"]), device=DEV)
    else:
        rows, n = c["M"], c["N"]
        s["y"] = torch.empty((c["M"], c["N"]), device=DEV)
    s["x"] = _normal(g, rows, c["K"]).to(DTYPES[c.get("dtype", "f32")])
    s["w"] = _weights(g, n, c["K"])
    if own:
        from block_quantized_matrix_amd import bqm

        s["wp"] = bqm.repack("mxfp4", s["w"].reshape(-1), n, c["K"])
        if c["op"] != "qmv":
            s["xp"] = _room(rows, c["K"])
    return s


def _room(rows, K):
    from block_quantized_matrix_amd import bqm

    return torch.empty(bqm.packed_bytes("mxfp4", rows, K), dtype=torch.uint8, device=DEV)


# ---- the plain forms ----

def _scale(e):
    """2^(e - 127) of e8m0 bytes, from the bits of a float; 255 stands for NaN."""
    e = e.to(torch.int32)
    bits = torch.where(e == 0, torch.full_like(e, 1 << 22), e << 23)
    return torch.where(e == 255, torch.full_like(e, 0x7FC00000), bits).view(torch.float32)


def _decode(blocks):
    """Interchange blocks [rows, nb, 17] -> fp32 [rows, 32 nb]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=blocks.device)
    codes = torch.cat([blocks[..., 1:] & 15, blocks[..., 1:] >> 4], -1)
    return (table[codes.to(torch.int32)] * _scale(blocks[..., :1])).reshape(blocks.shape[0], -1)


def _rounded(x):
    """x as MXFP4 holds it, fp32: blocks of 32 under the scale 2^(floor(log2 max) - 2), each value rounded to the
    nearest of the sixteen (ties to the even code) and kept within 6; a block that holds an infinity or a NaN is NaN."""
    v = x.to(torch.float32).reshape(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, torch.full_like(top, -127, dtype=torch.int32)).clamp_(min=-127)
    q = torch.ldexp(v.double(), -e).clamp(-6.0, 6.0)
    a = q.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    r = torch.round(q / step) * step * _scale(e + 127)
    return torch.where(torch.isfinite(top), r, math.nan).to(torch.float32).reshape(x.shape)


def _route(logits, bias, c):
    """Scores in 64 bits, since two experts next to each other decide an id. The ordering value is the logit itself where
    there is no bias (both scores grow with it)."""
    l = logits.double()
    score = torch.softmax(l, -1) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
    value = l if bias is None else score + bias.double()
    out = l == -math.inf
    value = torch.where(out, -math.inf, value)
    if c["n_group"] > 1:
        G, size = c["n_group"], c["E"] // c["n_group"]
        if c["group_top"] == 1:
            g = value.reshape(-1, G, size).amax(-1)
        else:
            whole = value if bias is not None else torch.where(out, -math.inf, score)
            two = whole.reshape(-1, G, size).sort(dim=-1, descending=True)[0][..., :2]
            g = two[..., 0] + torch.where(two[..., 1] == -math.inf, 0.0, two[..., 1])
        kept = g.sort(dim=-1, descending=True, stable=True)[1][:, :c["topk_group"]]
        open_ = torch.zeros_like(g, dtype=torch.bool).scatter_(1, kept, True)
        value = torch.where(open_.repeat_interleave(size, 1), value, -math.inf)
    best, ids = (t[:, :c["top_k"]] for t in value.sort(dim=-1, descending=True, stable=True))
    w = torch.where(best == -math.inf, 0.0, score.gather(1, ids))
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    return {"ids": torch.where(best == -math.inf, -1, ids).to(torch.int32), "weights": w.to(torch.float32)}


def _plain(s):
    c = s["case"]
    if c["op"] == "route":
        return _route(s["logits"], s["bias"], c)
    if c["op"] == "quantize":
        return _rounded(s["x"]).to(s["x"].dtype)
    if c["op"] == "qmv":
        return s["x"] @ _decode(s["w"]).t()
    if c["op"] == "qmm":
        return _rounded(s["x"]) @ _decode(s["w"]).t()
    y = (_rounded(s["x"]) @ _decode(s["w"]).t()).reshape(-1, c["E"], c["N"])  # every expert on every row
    slot = torch.arange(c["T"] * c["top_k"], device=DEV)
    row = slot if c["per_slot"] else slot // c["top_k"]
    return y[row, s["ids"].reshape(-1).long()].reshape(c["T"], c["top_k"], c["N"])


def _calls(s):
    from block_quantized_matrix_amd import bqm

    c = s["case"]
    if c["op"] == "route":
        bqm.bqm_route(c["score"], s["logits"], c["E"], s["bias"], c["T"], c["E"], c["n_group"], c["topk_group"],
                      c["group_top"], c["top_k"], c["renorm"], 1.0, s["ids"], s["weights"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if c["op"] == "qmv":
        bqm.qmv_mxfp4(s["wp"], s["x"], s["y"], c["M"], c["N"], c["K"])
        return s["y"]
    rows, K = s["x"].shape
    bqm.bqm_quantize_mxfp4(s["x"], K, s["xp"], rows, K)
    if c["op"] == "quantize":
        bqm.bqm_dequantize_mxfp4(s["xp"], s["y"], K, rows, K)
    elif c["op"] == "qmm":
        bqm.qmm_mxfp4(s["wp"], s["xp"], s["y"], rows, c["N"], K)
    else:
        bqm.qmm_id_mxfp4(s["wp"], c["E"], c["N"], K, s["ids"], c["T"], c["top_k"], s["xp"], rows,
                         c["top_k"] if c["per_slot"] else 1, 1 if c["per_slot"] else 0, s["y"])
    return s["y"]


def run(state):
    return _calls(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2}[c.get("dtype", "f32")]
    if c["op"] == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * size + (4 * c["E"] if c["bias"] else 0) + 8 * c["T"] * c["top_k"], "flops": 4 * n}
    if c["op"] == "quantize":
        return {"bytes": 2 * c["rows"] * c["K"] * size, "flops": 3 * c["rows"] * c["K"]}
    if c["op"] == "qmm_id":
        slots = c["T"] * c["top_k"]
        rows = slots if c["per_slot"] else c["T"]
        used = c["E"] * (1 - (1 - 1 / c["E"]) ** slots)  # experts that slots dealt evenly would reach
        return {"bytes": used * c["N"] * c["K"] * 17 / 32 + rows * c["K"] * size + 4 * slots * (c["N"] + 1),
                "flops": 2 * slots * c["N"] * c["K"]}
    return {"bytes": c["N"] * c["K"] * 17 / 32 + c["M"] * c["K"] * size + 4 * c["M"] * c["N"],
            "flops": 2 * c["M"] * c["N"] * c["K"]}


# ---- the definitions in 64 bits ----

def _exact_weights(blocks):
    b = blocks.to(torch.int64)
    nibble = torch.cat([b[..., 1:] % 16, b[..., 1:] // 16], -1)
    expo, frac = (nibble % 8) // 2, (nibble % 2).double()
    size = torch.where(expo == 0, frac * 0.5, (1 + frac / 2) * torch.ldexp(torch.ones_like(frac), expo - 1))
    return ((1 - 2 * (nibble // 8)) * torch.ldexp(size, b[..., :1] - 127)).reshape(blocks.shape[0], -1)


def _exact_rounded(x):
    """By distance: the value of the grid that is nearest, and of two as near the one with an even code."""
    v = x.double().reshape(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top)), torch.full_like(top, -125.0))
    e = e + (torch.pow(2.0, e + 1) <= top).double() - ((torch.pow(2.0, e) > top) & (top > 0)).double()
    unit = torch.pow(2.0, (e - 2).clamp(min=-127.0))
    a = v.abs() / unit
    best, away = torch.zeros_like(a), a.clone()
    for code, grid in enumerate(E2M1):
        d = (a - grid).abs()
        take = (d < away) | ((d == away) & (code % 2 == 0))
        best, away = torch.where(take, grid, best), torch.where(take, d, away)
    return (torch.sign(v) * best * unit).reshape(x.shape)


def _exact_route(logits, bias, c):
    """By counting: an expert's place is the number of those before it."""
    l = logits.double()
    if c["score"] == "softmax":
        z = torch.exp(l - l.amax(-1, keepdim=True))
        score = z / z.sum(-1, keepdim=True)
    else:
        score = torch.sigmoid(l)
    value = score + bias.double() if bias is not None else l

    def place(v):
        n, at = v.shape[1], torch.arange(v.shape[1], device=v.device)
        piece = max(1, (1 << 27) // (n * n))
        return torch.cat([((p[:, None, :] > p[:, :, None])
                           | ((p[:, None, :] == p[:, :, None]) & (at[None, :] < at[:, None]))).sum(-1)
                          for p in v.split(piece)])

    size = c["E"] // c["n_group"]
    if c["n_group"] > 1:
        v = value if c["group_top"] == 1 or bias is not None else score
        v = v.reshape(-1, c["n_group"], size)
        group = v.topk(c["group_top"], -1)[0].sum(-1)
        value = torch.where((place(group) < c["topk_group"]).repeat_interleave(size, 1), value, -math.inf)
    w = torch.zeros((l.shape[0], max(c["E"], c["top_k"])), dtype=torch.float64, device=l.device)
    w = w.scatter_(1, place(value), score)[:, :c["top_k"]]
    return {"ids": None, "weights": w / w.sum(-1, keepdim=True) if c["renorm"] else w}


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "route":
        return _exact_route(s["logits"], s["bias"], c)
    if c["op"] == "quantize":
        return _exact_rounded(s["x"])
    x = s["x"].double() if c["op"] == "qmv" else _exact_rounded(s["x"])
    n, chunk = s["w"].shape[0], max(1, (1 << 27) // c["K"])
    y = torch.cat([x @ _exact_weights(s["w"][r:r + chunk]).t() for r in range(0, n, chunk)], 1)
    if c["op"] != "qmm_id":
        return y
    y = y.reshape(y.shape[0], c["E"], c["N"])
    rows = torch.arange(c["T"] * c["top_k"], device=DEV).reshape(c["T"], c["top_k"])
    rows = rows if c["per_slot"] else rows // c["top_k"]
    return y[rows, s["ids"].long()]

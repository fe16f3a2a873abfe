"""Products of block-quantized weights with float rows, and the rows of a quantized table, in plain torch and as the
calls of block_quantized_matrix_amd.

Three operators, over weights in any of the block formats (Q4_0, Q8_0, MXFP4):

- embed: rows of a table by token id, times a scale (bqm_embed);
- linear: y = act(x W^T + bias) * mul + residual, one call from one token to long prompts (bqm_linear);
- grouped: the same where runs of rows, of any lengths, belong to the experts of a stacked W (bqm_linear_grouped).

Rows x, mul, residual and y are fp32, fp16 or bf16 and may lie apart by more than their length; bias is fp32.  mul makes
a gated feed-forward of it: silu(x Wg^T) * (x Wu^T).

Weights come as interchange blocks of 32: Q4_0 (18 bytes: binary16 d, then 16 bytes of which byte j holds code j in its
low nibble and code j + 16 in its high one; weight (code - 8) d), Q8_0 (34 bytes: d, then 32 signed codes; weight code d),
MXFP4 (17 bytes: e8m0 scale, then nibbles as for Q4_0, each an e2m1 number).  A program repacks them once, when it loads
its model, and keeps them so.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK = {"q4_0": 18, "q8_0": 34, "mxfp4": 17}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _linear(name, fmt, M, N, K, x, y=None, **more):
    return dict(dict(name=name, op="linear", fmt=fmt, M=M, N=N, K=K, x=x, y=y or x, bias=False, act="none", mul=False,
                     residual=False, pad=0), **more)


def _grouped(name, fmt, T, E, top_k, N, K, x, y=None, **more):
    return dict(dict(name=name, op="grouped", fmt=fmt, T=T, E=E, top_k=top_k, N=N, K=K, x=x, y=y or x, bias=False,
                     act="none", mul=False, residual=False, pad=0), **more)


def listed():
    return [
        # the embedding of one token at the start of every decode step: pure latency
        dict(name="embed one token", op="embed", fmt="q8_0", T=1, rows=65536, K=4096, y="bf16", scaled=False, pad=0),
        # the embeddings of a long prompt, scaled by sqrt(K)
        dict(name="embed a prompt", op="embed", fmt="q4_0", T=16384, rows=65536, K=5120, y="bf16", scaled=True, pad=0),
        # the smallest decode product of the benchmark as an output projection: its result added to the residual
        _linear("linear 4096 x 4096, one token", "q4_0", 1, 4096, 4096, "bf16", residual=True),
        # gate and up of the 27B dense model stacked, one token
        _linear("linear 34816 x 5120, one token", "q8_0", 1, 34816, 5120, "bf16"),
        # down of the 27B dense model, a decode batch, with bias and residual
        _linear("linear 5120 x 17408, 8 tokens", "mxfp4", 8, 5120, 17408, "f16", bias=True, residual=True),
        # a short prompt at sizes that no tile divides, fp32 throughout, rows apart
        _linear("linear ragged", "mxfp4", 33, 1000, 4128, "f32", bias=True, act="gelu", pad=24),
        # the 512-token prefill of the benchmark
        _linear("linear 512 tokens", "q8_0", 512, 17408, 5120, "bf16", act="silu"),
        # gate of the 27B dense model over a long prompt, times up's rows
        _linear("linear 4096 tokens", "q4_0", 4096, 17408, 5120, "bf16", act="silu", mul=True),
        # gate of the 128-expert layer, one token: eight experts' matrices, one row each
        _grouped("grouped one token", "q4_0", 1, 128, 8, 1536, 4096, "bf16", act="silu", mul=True),
        # down of the 128-expert layer over a batch of 64 tokens: about five rows an expert
        _grouped("grouped 64 tokens", "mxfp4", 64, 128, 8, 4096, 1536, "bf16", y="f32"),
        # gate over a 512-token prompt with a skewed router
        _grouped("grouped 512 tokens", "q4_0", 512, 128, 8, 1536, 4096, "bf16", act="silu", mul=True),
        # up over a long prompt
        _grouped("grouped 4096 tokens", "q8_0", 4096, 128, 8, 1536, 4096, "f16", bias=True),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["embed", "linear", "linear", "grouped", "grouped"])
    c = dict(op=op, fmt=rng.choice(list(BLOCK)), pad=rng.choice([0, 0, 0, 8, 40]))
    K = c["K"] = 32 * _log(rng, 1, 544)
    c["y"] = rng.choice(list(DTYPES))
    if op == "embed":
        return dict(c, T=_log(rng, 1, min(16384, 16384 * 5120 // K)), rows=_log(rng, 100, min(262144, 65536 * 5120 // K)),
                    scaled=rng.random() < 0.5)
    c["x"] = rng.choice(["bf16", "f16", "f32"])
    if rng.random() < 0.7:
        c["y"] = c["x"]
    c.update(bias=rng.random() < 0.4, act=rng.choice(ACTS), mul=rng.random() < 0.3, residual=rng.random() < 0.4)
    if op == "linear":
        return dict(c, M=_log(rng, 1, 4096), N=_log(rng, 16, min(34816, 17408 * 5120 // K)))
    E = _log(rng, 4, 128)
    N = _log(rng, 16, min(4096, 1536 * 4096 * 128 // (K * E)))
    return dict(c, T=_log(rng, 1, min(4096, 4096 * 1536 * 4096 // (N * K))), E=E, top_k=rng.randint(1, min(8, E)), N=N)


# ---- inputs ----

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _half_bytes(d):
    return d.reshape(d.shape[0], -1, 1).view(torch.uint8)


def _blocks(fmt, w):
    """Interchange blocks [rows, K/32, bytes] of float rows, as a checkpoint holds them."""
    v = w.reshape(w.shape[0], -1, 32)
    top = v.abs().amax(-1)
    if fmt == "q8_0":
        d = (top / 127).to(torch.float16)
        code = torch.round(v / d.float().clamp(min=1e-7)[..., None]).clamp_(-127, 127).to(torch.int8)
        return torch.cat([_half_bytes(d), code.view(torch.uint8)], -1)
    if fmt == "q4_0":
        most = torch.gather(v, -1, v.abs().argmax(-1, keepdim=True))[..., 0]
        d = (most / -8).to(torch.float16)
        f = torch.where(d == 0, torch.ones_like(d), d).float()[..., None]
        code = (torch.round(v / f) + 8).clamp_(0, 15).to(torch.uint8)
        return torch.cat([_half_bytes(d), code[..., :16] | (code[..., 16:] << 4)], -1)
    e = torch.frexp(top[..., None])[1].clamp_(min=-124, max=130) + 124
    q = v * torch.pow(2.0, (127 - e).to(torch.float32))
    a = q.abs()
    code = torch.zeros_like(v, dtype=torch.uint8)
    for edge in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):  # weights on an edge itself do not occur in earnest
        code += a > edge
    code += (q < 0).to(torch.uint8) * 8
    return torch.cat([e.to(torch.uint8), code[..., :16] | (code[..., 16:] << 4)], -1)


def _weights(g, fmt, rows, K):
    """Blocks of normal weights, made in pieces that keep the floats small."""
    piece = max(1, (1 << 27) // K)
    return torch.cat([_blocks(fmt, _normal(g, min(piece, rows - r), K) * 0.02) for r in range(0, rows, piece)])


def _rows(g, n, width, pad, dtype):
    """n rows of normal numbers, pad elements apart."""
    return _normal(g, n, width + pad).to(DTYPES[dtype])[:, :width]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, s = case, {"case": case}
    y = DTYPES[c["y"]]
    if c["op"] == "embed":
        rows, M, N, K = c["rows"], c["T"], c["K"], c["K"]
        s["ids"] = torch.randint(0, rows, (M,), generator=g, device=DEV, dtype=torch.int32)
        s["scale"] = torch.tensor(math.sqrt(K) if c["scaled"] else 1.0).item()  # a number of fp32
    else:
        N, K = c["N"], c["K"]
        rows, M = (N, c["M"]) if c["op"] == "linear" else (c["E"] * N, c["T"] * c["top_k"])
        s["x"] = _rows(g, M, K, c["pad"], c["x"])
        s["bias"] = _normal(g, rows) * 0.1 if c["bias"] else None
        s["mul"] = _rows(g, M, N, c["pad"], c["y"]) if c["mul"] else None
        s["residual"] = _rows(g, M, N, c["pad"], c["y"]) if c["residual"] else None
    if c["op"] == "grouped":  # rows in the order of the experts that a skewed router chose
        logits = _normal(g, c["T"], c["E"]) - 1.1 * torch.arange(1, c["E"] + 1, device=DEV).log()
        ids = logits.argsort(-1, descending=True)[:, :c["top_k"]].reshape(-1)
        counts = torch.bincount(ids, minlength=c["E"])
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["ends"] = s["offsets"].tolist()
    s["out"] = torch.empty((M, N + c["pad"]), dtype=y, device=DEV)[:, :N]
    s["w"] = _weights(g, c["fmt"], rows, K)
    if own:
        from block_quantized_matrix_amd import bqm

        s["wp"] = bqm.repack(c["fmt"], s["w"].reshape(-1), rows, K)
    return s


# ---- the plain forms ----

def _scale(e):
    """2^(e - 127) of e8m0 bytes, from the bits of a float; 255 stands for NaN."""
    e = e.to(torch.int32)
    bits = torch.where(e == 0, torch.full_like(e, 1 << 22), e << 23)
    return torch.where(e == 255, torch.full_like(e, 0x7FC00000), bits).view(torch.float32)


def _decode(fmt, blocks):
    """Interchange blocks [rows, nb, bytes] -> fp32 [rows, 32 nb], exact."""
    if fmt == "mxfp4":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=blocks.device)
        codes = torch.cat([blocks[..., 1:] & 15, blocks[..., 1:] >> 4], -1)
        return (table[codes.to(torch.int32)] * _scale(blocks[..., :1])).reshape(blocks.shape[0], -1)
    d = blocks[..., :2].contiguous().view(torch.float16).float()
    body = blocks[..., 2:]
    if fmt == "q8_0":
        codes = body.contiguous().view(torch.int8).float()
    else:
        codes = torch.cat([body & 15, body >> 4], -1).float() - 8.0
    return (codes * d).reshape(blocks.shape[0], -1)


def _act(name, z):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _finish(s, z):
    c = s["case"]
    z = _act(c["act"], z)
    if s["mul"] is not None:
        z = z * s["mul"].float()
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(DTYPES[c["y"]])


def _plain(s):
    c = s["case"]
    if c["op"] == "embed":
        return (_decode(c["fmt"], s["w"][s["ids"].long()]) * s["scale"]).to(DTYPES[c["y"]])
    if c["op"] == "linear":
        z = s["x"].float() @ _decode(c["fmt"], s["w"]).t()
        return _finish(s, z if s["bias"] is None else z + s["bias"])
    E, N, ends = c["E"], c["N"], s["ends"]
    z = torch.empty((ends[E], N), device=DEV)
    for e in range(E):
        if ends[e] < ends[e + 1]:
            p = s["x"][ends[e]:ends[e + 1]].float() @ _decode(c["fmt"], s["w"][e * N:(e + 1) * N]).t()
            z[ends[e]:ends[e + 1]] = p if s["bias"] is None else p + s["bias"][e * N:(e + 1) * N]
    return _finish(s, z)


def _calls(s):
    from block_quantized_matrix_amd import bqm

    c, y = s["case"], s["out"]
    if c["op"] == "embed":
        bqm.bqm_embed(c["fmt"], s["wp"], c["rows"], c["K"], s["ids"], c["T"], s["scale"], y, y.stride(0))
        return y
    mul, res = s["mul"], s["residual"]
    more = dict(bias=s["bias"], act=c["act"], mul=mul, mul_stride=0 if mul is None else mul.stride(0), residual=res,
                res_stride=0 if res is None else res.stride(0))
    if c["op"] == "linear":
        bqm.bqm_linear(c["fmt"], s["wp"], s["x"], s["x"].stride(0), y, y.stride(0), c["M"], c["N"], c["K"], **more)
    else:
        bqm.bqm_linear_grouped(c["fmt"], s["wp"], c["E"], s["offsets"], s["x"], s["x"].stride(0), y, y.stride(0),
                               c["T"] * c["top_k"], c["N"], c["K"], **more)
    return y


def run(state):
    return _calls(state) if own else _plain(state)


# ---- what a pass cannot do without ----

def work(case):
    c = case
    size = {"f32": 4, "f16": 2, "bf16": 2}
    block = BLOCK[c["fmt"]] / 32
    if c["op"] == "embed":
        return {"bytes": c["T"] * (c["K"] * (block + size[c["y"]]) + 4), "flops": 2 * c["T"] * c["K"]}
    N, K = c["N"], c["K"]
    M = c["M"] if c["op"] == "linear" else c["T"] * c["top_k"]
    matrices = 1 if c["op"] == "linear" else c["E"] * (1 - (1 - 1 / c["E"]) ** M)  # that rows dealt evenly would reach
    return {"bytes": matrices * (N * K * block + (4 * N if c["bias"] else 0)) + M * K * size[c["x"]]
            + (1 + c["mul"] + c["residual"]) * M * N * size[c["y"]], "flops": 2 * M * N * K}


# ---- the definitions in 64 bits ----

def _exact_weights(fmt, blocks):
    b = blocks.to(torch.int64)
    rows, nb = b.shape[:2]
    if fmt == "q8_0":
        w = (b[..., 2:] + 128) % 256 - 128
    else:
        w = torch.zeros((rows, nb, 32), dtype=torch.int64, device=b.device)
        w[..., :16] = b[..., -16:] % 16
        w[..., 16:] = b[..., -16:] // 16
    if fmt == "mxfp4":
        expo, frac = (w % 8) // 2, (w % 2).double()
        size = torch.where(expo == 0, frac * 0.5, (1 + frac / 2) * torch.ldexp(torch.ones_like(frac), expo - 1))
        return ((1 - 2 * (w // 8)) * torch.ldexp(size, b[..., :1] - 127)).reshape(rows, -1)
    h = b[..., :1] + 256 * b[..., 1:2]  # binary16 from its fields
    expo, frac = h // 1024 % 32, (h % 1024).double()
    d = torch.where(expo == 0, torch.ldexp(frac, torch.full_like(expo, -24)), torch.ldexp(1024 + frac, expo - 25))
    return ((w - (8 if fmt == "q4_0" else 0)) * (1 - 2 * (h // 32768)) * d).reshape(rows, -1)


def _exact_product(c, x, blocks):
    chunk = max(1, (1 << 27) // c["K"])
    return torch.cat([x @ _exact_weights(c["fmt"], blocks[r:r + chunk]).t() for r in range(0, blocks.shape[0], chunk)], 1)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "embed":
        ids, piece = s["ids"].long(), max(1, (1 << 26) // c["K"])
        return torch.cat([_exact_weights(c["fmt"], s["w"][i]) for i in ids.split(piece)]) * s["scale"]
    x = s["x"].double()
    if c["op"] == "linear":
        z = _exact_product(c, x, s["w"])
        if c["bias"]:
            z += s["bias"].double()
    else:
        w = s["w"].reshape(c["E"], c["N"], *s["w"].shape[1:])
        parts = []
        for e, (i, j) in enumerate(zip(s["ends"], s["ends"][1:])):
            if j > i:
                z = _exact_product(c, x[i:j], w[e])
                parts.append(z + s["bias"].double().reshape(c["E"], -1)[e] if c["bias"] else z)
        z = torch.cat(parts)
    if c["act"] == "relu":
        z = z.clamp(min=0)
    elif c["act"] == "silu":
        z = z * torch.sigmoid(z)
    elif c["act"] == "gelu":
        z = z * torch.special.ndtr(z)
    elif c["act"] == "gelu_tanh":
        z = z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
    if c["mul"]:
        z = z * s["mul"].double()
    return z + s["residual"].double() if c["residual"] else z

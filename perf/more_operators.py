"""Operators on the rows between products, as measured cases: layer norm with dropout and residual
add in front of it (forward and backward), dropout from a counter-based generator, int8 codes with a
scale per row, and the product of int8 codes with scales per token and per channel.

``run`` computes an operator's plain form with elementary torch operations, or, with ``own`` set, makes
the calls a program makes of ``gemm_epilogue_transformer_tiled_amd.rows``.

    norm      s = R + drop(X), as stored; n = (s - mean) / sqrt(var + eps); y = n * gain + bias
              e = dY * gain; g = rstd * (e - mean(e) - n * mean(e n)) + dS; dR = g; dX = drop(g);
              dgain = sum over rows of dY n; dbias = sum over rows of dY
    dropout   value j of the row's block b of eight has half-word j of the four words of Philox4x32-10
              with key seed and counter (row * ceil(d / 8) + b, site, offset, offset >> 32); it is dropped
              where that is below t = round(p 2^16), and times 2^16 / (2^16 - t) elsewhere
    quant     scale = max|x| / 127 of a row, code = 127 x / max|x| to nearest, ties to even
    int8      Y = act(x_scale[m] * w_scale[n] * sum_k X[m, k] W[n, k] + bias[n]) + R
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
EPS = 1e-5


def listed():
    return [
        # serving: the norm before a block for 16 sequences' tokens, residual added on the way
        {"name": "norm decode", "op": "norm_fwd", "M": 16, "d": 4096, "dtype": "bf16", "residual": True, "p": 0.0},
        # training: 16384 tokens, dropout on the block's output, residual added, statistics kept
        {"name": "norm train forward", "op": "norm_fwd", "M": 16384, "d": 4096, "dtype": "bf16", "residual": True,
         "p": 0.1},
        # its gradient, with the gradient that arrives on the residual stream
        {"name": "norm train backward", "op": "norm_bwd", "M": 16384, "d": 4096, "dtype": "bf16", "residual": True,
         "p": 0.1},
        # fine-tuning in 32 bits on one odd sequence, a width that is no multiple of anything
        {"name": "norm odd backward", "op": "norm_bwd", "M": 1001, "d": 1021, "dtype": "fp32", "residual": False, "p": 0.0},
        # training: dropout of a feed-forward block's hidden values
        {"name": "dropout hidden", "op": "dropout", "M": 8192, "d": 11008, "dtype": "bf16", "residual": False, "p": 0.1},
        # dropout and residual add in 32 bits, odd sizes
        {"name": "dropout odd", "op": "dropout", "M": 777, "d": 1021, "dtype": "fp32", "residual": True, "p": 0.25},
        # serving: the codes of a decoding batch's tokens
        {"name": "quant decode", "op": "quant", "M": 27, "d": 4096, "dtype": "bf16"},
        # the codes of a prompt's hidden values
        {"name": "quant prompt", "op": "quant", "M": 8192, "d": 11008, "dtype": "bf16"},
        # serving: one token through the up projection
        {"name": "int8 one token", "op": "int8", "M": 1, "N": 11008, "K": 4096, "act": "none", "bias": False,
         "residual": False, "dtype": "bf16"},
        # a decoding batch of odd size through the down projection, residual added
        {"name": "int8 decode batch", "op": "int8", "M": 27, "N": 4096, "K": 11008, "act": "none", "bias": False,
         "residual": True, "dtype": "bf16"},
        # a ragged prompt through a smaller layer, no size a multiple of a tile
        {"name": "int8 ragged prompt", "op": "int8", "M": 777, "N": 2856, "K": 1040, "act": "gelu_tanh", "bias": True,
         "residual": False, "dtype": "fp32"},
        # a prompt of 8192 tokens at the widths of the SwiGLU workload
        {"name": "int8 prompt", "op": "int8", "M": 8192, "N": 11008, "K": 4096, "act": "silu", "bias": True,
         "residual": False, "dtype": "bf16"},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` from lo to hi, even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "dropout", "quant", "int8", "int8"])
    if op == "int8":
        return {"op": op, "M": _spread(rng, 1, 8192), "N": _spread(rng, 256, 11008, 8), "K": _spread(rng, 256, 11008 // 16 * 16, 16)
                if rng.random() < 0.5 else _spread(rng, 256, 4096, 64), "act": rng.choice(["none", "silu", "gelu_tanh", "relu"]),
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5, "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    size = 2 if dtype == "bf16" else 4
    # widths: rows that start anywhere, whole vectors, whole lines
    d = _spread(rng, 64, 11008, rng.choice([1, 8, 64]))
    M = _spread(rng, 1, max(2, min(16384, 16384 * 4096 * 2 // (d * size))))
    c = {"op": op, "M": M, "d": d, "dtype": dtype}
    if op != "quant":
        c.update(residual=rng.random() < 0.5, p=rng.choice([0.0, 0.1, 0.1, 0.5]) if op != "dropout" else rng.choice([0.05, 0.1, 0.5]))
    return c


# ---- inputs ----

def _normal(gen, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32) * std).to(dtype)


def _type(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _stream(gen, M, d, dtype):
    """Rows of a residual stream: a few channels are far larger than the others."""
    x = torch.randn((M, d), generator=gen, device=DEVICE)
    x[:, d // 3::997] *= 20.0
    return (x + 0.1).to(dtype)


def _rng(seed, p):
    """Seed and offset of the generator, on the GPU as a program keeps them; site: which dropout of a step."""
    return torch.tensor([0x9E3779B97F4A7C15 * (seed + 1) % (1 << 62), (1 << 33) + 7 * seed], dtype=torch.int64,
                        device=DEVICE) if p else None


def _prepare_norm(c, gen, seed):
    M, d, dtype, p = c["M"], c["d"], _type(c), c["p"]
    s = {"gain": (1 + 0.1 * torch.randn(d, generator=gen, device=DEVICE)).to(dtype), "bias": _normal(gen, (d,), 0.1, dtype),
         "rng": _rng(seed, p), "site": 3}
    kept = c["residual"] or p > 0                      # the sum is a tensor of its own
    if c["op"] == "norm_fwd":
        s["X"] = _normal(gen, (M, d), 1.0, dtype) if c["residual"] else _stream(gen, M, d, dtype)
        s["R"] = _stream(gen, M, d, dtype) if c["residual"] else None
    else:
        s["S"] = _stream(gen, M, d, dtype)
        x = s["S"].double()
        mean = x.mean(-1)
        s["mean"], s["rstd"] = mean.float(), torch.rsqrt((x - mean[:, None]).square().mean(-1) + EPS).float()
        s["dY"] = _normal(gen, (M, d), 0.02, dtype)
        s["dS"] = _normal(gen, (M, d), 0.02, dtype) if kept else None
    if own:
        from gemm_epilogue_transformer_tiled_amd import rows
        s["plan"] = rows.LayerNorm(M, d, eps=EPS, dtype=dtype, residual=c["residual"], dropout=p, site=s["site"])
        new = lambda: torch.empty((M, d), dtype=dtype, device=DEVICE)  # noqa: E731
        if c["op"] == "norm_fwd":
            s["out"] = {"Y": new(), "mean": torch.empty(M, device=DEVICE), "rstd": torch.empty(M, device=DEVICE)}
            if kept:
                s["out"]["S"] = new()
            s["args"] = rows.make_norm_args(X=s["X"], residual=s["R"], gain=s["gain"], bias=s["bias"], rng=s["rng"], **s["out"])
        else:
            s["out"] = {"dX": new(), "dgain": torch.empty(d, device=DEVICE), "dbias": torch.empty(d, device=DEVICE)}
            if c["residual"] and p > 0:
                s["out"]["dR"] = new()
            s["args"] = rows.make_norm_args(S=s["S"], mean=s["mean"], rstd=s["rstd"], gain=s["gain"], rng=s["rng"], dY=s["dY"],
                                            dS=s["dS"], **s["out"])
    return s


def _prepare_dropout(c, gen, seed):
    M, d, dtype = c["M"], c["d"], _type(c)
    s = {"X": _normal(gen, (M, d), 1.0, dtype), "R": _stream(gen, M, d, dtype) if c["residual"] else None,
         "rng": _rng(seed, c["p"]), "site": 5}
    if own:
        from gemm_epilogue_transformer_tiled_amd import rows
        s["plan"] = rows.Dropout(M, d, c["p"], dtype=dtype, residual=c["residual"], site=s["site"])
        s["out"] = {"Y": torch.empty((M, d), dtype=dtype, device=DEVICE)}
        s["args"] = rows.make_dropout_args(X=s["X"], residual=s["R"], rng=s["rng"], **s["out"])
    return s


def _prepare_quant(c, gen, seed):
    M, d, dtype = c["M"], c["d"], _type(c)
    s = {"X": _stream(gen, M, d, dtype)}
    if own:
        from gemm_epilogue_transformer_tiled_amd import rows
        s["plan"] = rows.RowQuant(M, d, dtype=dtype)
        s["out"] = {"codes": torch.empty((M, d), dtype=torch.int8, device=DEVICE), "scale": torch.empty(M, device=DEVICE)}
        s["args"] = rows.make_quant_args(X=s["X"], **s["out"])
    return s


def _codes(gen, n, k, std):
    """int8 codes of normal rows and their scales."""
    w = torch.randn((n, k), generator=gen, device=DEVICE) * std
    scale = w.abs().amax(-1) / 127.0
    return torch.round(w / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def _prepare_int8(c, gen, seed):
    M, N, K, dtype = c["M"], c["N"], c["K"], _type(c)
    s = {}
    s["X"], s["x_scale"] = _codes(gen, M, K, 1.0)
    s["W"], s["w_scale"] = _codes(gen, N, K, K ** -0.5)
    s["bias"] = _normal(gen, (N,), 0.5, dtype) if c["bias"] else None
    s["R"] = _normal(gen, (M, N), 1.0, dtype) if c["residual"] else None
    if own:
        from gemm_epilogue_transformer_tiled_amd import rows
        s["plan"] = rows.Int8Linear(M, N, K, act=c["act"], bias=c["bias"], residual=c["residual"], dtype=dtype)
        s["out"] = {"Y": torch.empty((M, N), dtype=dtype, device=DEVICE)}
        s["args"] = rows.make_i8_args(X=s["X"], W=s["W"], x_scale=s["x_scale"], w_scale=s["w_scale"], bias=s["bias"],
                                      residual=s["R"], **s["out"])
    return s


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    make = {"norm_fwd": _prepare_norm, "norm_bwd": _prepare_norm, "dropout": _prepare_dropout, "quant": _prepare_quant,
            "int8": _prepare_int8}[case["op"]]
    s = make(case, gen, seed)
    s["case"] = case
    return s


# ---- plain forms ----

_LOW = 0xFFFFFFFF


def _keep(s, M, d):
    """(which values are kept, their factor): Philox4x32-10 in 64-bit integers."""
    t = int(round(s["case"]["p"] * 65536))
    blocks = (d + 7) // 8
    seed, offset = s["rng"][0], s["rng"][1]
    c0 = torch.arange(M * blocks, device=DEVICE, dtype=torch.int64)
    c1 = torch.full_like(c0, s["site"])
    c2, c3 = (offset & _LOW).expand_as(c0), ((offset >> 32) & _LOW).expand_as(c0)
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for i in range(10):
        if i:
            k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
        # products of 32-bit values: the low 64 bits are right whatever their sign
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW
    words = torch.stack([c0, c1, c2, c3], -1)
    half = torch.stack([words & 0xFFFF, words >> 16], -1).view(M, blocks * 8)[:, :d]
    return half >= t, 65536.0 / (65536 - t)


def _drop(s, x):
    """x in 32 bits with values dropped, or x itself where nothing is."""
    if not s["case"]["p"]:
        return x
    keep, factor = _keep(s, *x.shape)
    return torch.where(keep, x * factor, torch.zeros((), device=DEVICE))


def _plain_norm_fwd(s):
    c, X = s["case"], s["X"]
    out = {}
    x = _drop(s, X.float())
    if c["residual"]:
        x = s["R"].float() + x
    if c["residual"] or c["p"]:
        out["S"] = x.to(X.dtype)
        x = out["S"].float()                           # the norm of the sum as it is kept
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + EPS)
    y = (x - mean) * rstd * s["gain"].float() + s["bias"].float()
    out.update(Y=y.to(X.dtype), mean=mean[:, 0], rstd=rstd[:, 0])
    return out


def _plain_norm_bwd(s):
    c, x, dy = s["case"], s["S"].float(), s["dY"].float()
    n = (x - s["mean"][:, None]) * s["rstd"][:, None]
    e = dy * s["gain"].float()
    g = s["rstd"][:, None] * (e - e.mean(-1, keepdim=True) - n * (e * n).mean(-1, keepdim=True))
    if s["dS"] is not None:
        g = g + s["dS"].float()
    out = {"dX": _drop(s, g).to(s["S"].dtype), "dgain": (dy.double() * n.double()).sum(0).float(),
           "dbias": dy.double().sum(0).float()}
    if c["residual"] and c["p"]:
        out["dR"] = g.to(s["S"].dtype)
    return out


def _plain_dropout(s):
    y = _drop(s, s["X"].float())
    if s["R"] is not None:
        y = s["R"].float() + y
    return {"Y": y.to(s["X"].dtype)}


def _plain_quant(s):
    # the exact quotient decides: 32-bit inputs need 64 bits next to a tie
    x = s["X"].double() if s["X"].dtype == torch.float32 else s["X"].float()
    top = x.abs().amax(-1)
    codes = torch.round(x * 127.0 / torch.where(top > 0, top, torch.ones_like(top))[:, None])
    return {"codes": codes.to(torch.int8), "scale": (top / 127.0).float()}


def _act(name, t):
    if name == "silu":
        return t / (1 + torch.exp(-t))
    if name == "relu":
        return t * (t > 0)
    if name == "gelu_tanh":
        return t / (1 + torch.exp(-2 * 0.7978845608028654 * (t + 0.044715 * t * t * t)))
    return t


def _plain_int8(s):
    t = (s["X"].float() @ s["W"].float().t()) * s["x_scale"][:, None] * s["w_scale"]
    if s["bias"] is not None:
        t = t + s["bias"].float()
    y = _act(s["case"]["act"], t)
    if s["R"] is not None:
        y = y + s["R"].float()
    return {"Y": y.to(_type(s["case"]))}


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "norm_bwd":
            s["plan"].backward(s["args"])
        elif op in ("norm_fwd", "dropout"):
            s["plan"].forward(s["args"])
        else:
            s["plan"].run(s["args"])
        return s["out"]
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "dropout": _plain_dropout, "quant": _plain_quant,
            "int8": _plain_int8}[op](s)


# ---- the definitions in 64 bits ----

def _factors(s, M, d):
    """What dropout multiplies each value with, 64 bits, on the host's 32 x 32 -> 64-bit products."""
    p = s["case"]["p"]
    if not p:
        return torch.ones((), dtype=torch.float64, device=DEVICE)
    seed, offset = (int(v) & (1 << 64) - 1 for v in s["rng"].cpu())
    nb = -(-d // 8)
    u32, u64, sh = np.uint32, np.uint64, np.uint64(32)
    ctr = [np.arange(M * nb, dtype=u32), np.full(M * nb, s["site"], u32), np.full(M * nb, offset & _LOW, u32),
           np.full(M * nb, offset >> 32, u32)]
    keys = [(u32((seed + r * 0x9E3779B9) & _LOW), u32(((seed >> 32) + r * 0xBB67AE85) & _LOW)) for r in range(10)]
    for k0, k1 in keys:
        p0, p1 = ctr[0].astype(u64) * u64(0xD2511F53), ctr[2].astype(u64) * u64(0xCD9E8D57)
        ctr = [(p1 >> sh).astype(u32) ^ ctr[1] ^ k0, p1.astype(u32), (p0 >> sh).astype(u32) ^ ctr[3] ^ k1, p0.astype(u32)]
    u = np.empty((M * nb, 8), np.uint16)
    for i, w in enumerate(ctr):
        u[:, 2 * i], u[:, 2 * i + 1] = w & u32(0xFFFF), w >> u32(16)
    t = math.floor(p * 65536 + 0.5)
    kept = torch.from_numpy(u.reshape(M, nb * 8)[:, :d] >= t).to(DEVICE)
    return kept.double() * (65536.0 / (65536 - t))


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "int8":
        t = torch.matmul(s["X"].to(f64), s["W"].to(f64).T)
        t = t.mul_(s["x_scale"].to(f64)[:, None]).mul_(s["w_scale"].to(f64))
        if case["bias"]:
            t += s["bias"].to(f64)
        if case["act"] == "silu":
            t = t * torch.special.expit(t)
        elif case["act"] == "relu":
            t = t.clamp(min=0)
        elif case["act"] == "gelu_tanh":
            t = 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))
        return {"Y": t + s["R"].to(f64) if case["residual"] else t}
    if op == "quant":
        x = s["X"].to(f64)
        a = torch.maximum(x.amax(1), -x.amin(1))
        q = 127 * x / a.clamp(min=torch.finfo(f64).tiny)[:, None]
        low = q.floor()
        up = (q - low > 0.5) | ((q - low == 0.5) & (low % 2 != 0))
        return {"codes": (low + up).to(torch.int8), "scale": a / 127}
    M, d = case["M"], case["d"]
    F = _factors(s, M, d)
    dtype = _type(case)
    if op == "dropout":
        y = F * s["X"].to(f64)
        return {"Y": y + s["R"].to(f64) if case["residual"] else y}
    if op == "norm_fwd":
        x = F * s["X"].to(f64)
        out = {}
        if case["residual"]:
            x = x + s["R"].to(f64)
        if case["residual"] or case["p"]:
            out["S"] = x
            x = x.to(dtype).to(f64)                    # what is normalised is the sum as it is kept
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = (var + EPS).pow(-0.5)
        return {"Y": torch.addcmul(s["bias"].to(f64), (x - mean) * rstd, s["gain"].to(f64)), "mean": mean.squeeze(1),
                "rstd": rstd.squeeze(1), **out}
    x, dy, r = s["S"].to(f64), s["dY"].to(f64), s["rstd"].to(f64)[:, None]
    xc = x - s["mean"].to(f64)[:, None]
    e = dy * s["gain"].to(f64)
    g = r * e - r * e.sum(1, keepdim=True) / d - xc * (r ** 3 * (e * xc).sum(1, keepdim=True) / d)
    if s["dS"] is not None:
        g += s["dS"].to(f64)
    out = {"dX": F * g, "dgain": (dy * xc * r).sum(0), "dbias": dy.sum(0)}
    if case["residual"] and case["p"]:
        out["dR"] = g
    return out


def work(case):
    op = case["op"]
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        # codes and scales read, Y written, R and the bias read
        return {"bytes": M * K + N * K + 4 * (M + N) + size * M * N * (2 if case["residual"] else 1) +
                (size * N if case["bias"] else 0), "flops": 2 * M * N * K}
    M, d = case["M"], case["d"]
    values = M * d
    if op == "quant":
        return {"bytes": values * (size + 1) + 4 * M, "flops": 4 * values}
    if op == "dropout":
        return {"bytes": size * values * (3 if case["residual"] else 2), "flops": 2 * values}
    kept = case["residual"] or case["p"] > 0
    if op == "norm_fwd":
        # X (and R) read, Y (and the kept sum) written, statistics written
        return {"bytes": size * (values * (2 + case["residual"] + kept) + 2 * d) + 8 * M, "flops": 8 * values}
    # dY, the kept sum (and the residual's gradient) read, dX (and dR) written, gains' gradients written
    both = case["residual"] and case["p"] > 0
    return {"bytes": size * (values * (3 + kept + both) + d) + 8 * M + 8 * d, "flops": 14 * values}

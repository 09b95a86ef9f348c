"""The transformer-block operators around the fused products, as measured cases: the gated
feed-forward block (forward and backward), the per-head norm of queries and keys with the position
rotation (forward and backward), and the global gradient norm with clipping.

``run`` computes an operator's plain form with elementary torch operations in 32 bits, or, with
``own`` set, makes the calls a program makes of ``gemm_epilogue_transformer_tiled_amd.block``.

    feed-forward  G = X Wg, U = X Wu, H = act(G) * U, Y = H Wd (+ R)
                  dH = dY Wd^T, dG = dH * U * act'(G), dU = dH * act(G)
                  dX = dG Wg^T + dU Wu^T, dWg = X^T dG, dWu = X^T dU, dWd = H^T dY
    norm + rotary per head of D values: n = x / sqrt(mean(x^2) + eps), y = n * gain; the first
                  `rot` values of y turn in pairs by position * inv_freq[i], times `amplitude`
    clipping      norm = sqrt(sum of all squares), every gradient times min(1, max / (norm + eps))
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
NORM_EPS = 1e-6
CLIP_EPS = 1e-6


def listed():
    return [
        # serving: one token through the block at the widths of the SwiGLU workload
        {"name": "ffn one token", "op": "ffn_fwd", "M": 1, "d": 4096, "h": 11008, "act": "silu", "layout": "kn",
         "residual": True, "save": False},
        # serving: a decoding batch of odd size, weights stored [out][in] as linear layers keep them
        {"name": "ffn decode batch", "op": "ffn_fwd", "M": 27, "d": 4096, "h": 11008, "act": "silu", "layout": "nk",
         "residual": True, "save": False},
        # a ragged prompt through a smaller block: no size a multiple of a tile
        {"name": "ffn ragged prompt", "op": "ffn_fwd", "M": 777, "d": 1032, "h": 2856, "act": "gelu_tanh",
         "layout": "kn", "residual": False, "save": True},
        # training: 8192 tokens, pre-activations kept for the backward pass
        {"name": "ffn train forward", "op": "ffn_fwd", "M": 8192, "d": 4096, "h": 11008, "act": "silu",
         "layout": "kn", "residual": True, "save": True},
        # fine-tuning on one short odd sequence
        {"name": "ffn short backward", "op": "ffn_bwd", "M": 333, "d": 1032, "h": 2856, "act": "silu", "layout": "nk"},
        # the training step's backward pass, all four gradients
        {"name": "ffn train backward", "op": "ffn_bwd", "M": 8192, "d": 4096, "h": 11008, "act": "silu",
         "layout": "kn"},
        # serving: one token for each of 16 sequences, each at its own far position
        {"name": "rotary decode", "op": "qk_fwd", "T": 16, "hq": 32, "hk": 8, "D": 128, "rot": 128, "pairs": "half",
         "norm": True, "dtype": "bf16", "far": 100000, "factor": 4.0},
        # a prompt of 16384 tokens, grouped heads, 128 values a head
        {"name": "rotary prompt", "op": "qk_fwd", "T": 16384, "hq": 32, "hk": 8, "D": 128, "rot": 128,
         "pairs": "half", "norm": True, "dtype": "bf16", "far": 0, "factor": 1.0},
        # its gradient
        {"name": "rotary train backward", "op": "qk_bwd", "T": 16384, "hq": 32, "hk": 8, "D": 128, "rot": 128,
         "pairs": "half", "norm": True, "dtype": "bf16", "far": 0, "factor": 1.0},
        # 32-bit values, interleaved pairs on part of the head, odd token count
        {"name": "rotary partial backward", "op": "qk_bwd", "T": 1001, "hq": 12, "hk": 12, "D": 80, "rot": 40,
         "pairs": "interleaved", "norm": True, "dtype": "fp32", "far": 30000, "factor": 1.0},
        # a small model's gradients of mixed types, packed without padding (odd addresses)
        {"name": "clip small", "op": "clip", "layers": 4, "d": 264, "h": 712, "mixed": True, "clips": True},
        # the feed-forward gradients of eight layers
        {"name": "clip large", "op": "clip", "layers": 8, "d": 4096, "h": 11008, "mixed": False, "clips": True},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` from lo to hi, even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_fwd", "ffn_bwd", "qk_fwd", "qk_bwd", "clip"])
    if op in ("ffn_fwd", "ffn_bwd"):
        d, h = _spread(rng, 256, 4096, 8), _spread(rng, 512, 11008, 8)
        M = _spread(rng, 1 if op == "ffn_fwd" else 16, 8192)
        c = {"op": op, "M": M, "d": d, "h": h, "act": rng.choice(["silu", "silu", "gelu_tanh", "relu"]),
             "layout": rng.choice(["kn", "nk"])}
        if op == "ffn_fwd":
            c.update(residual=rng.random() < 0.5, save=rng.random() < 0.5)
        return c
    if op in ("qk_fwd", "qk_bwd"):
        D = rng.choice([64, 80, 96, 128, 256])
        hk = rng.choice([1, 2, 8])
        hq = hk * rng.choice([1, 3, 4])
        most = max(2, min(16384, 16384 * 40 * 128 // ((hq + hk) * D)))
        return {"op": op, "T": _spread(rng, 1, most), "hq": hq, "hk": hk, "D": D,
                "rot": rng.choice([D, D, D // 2, D // 4]), "pairs": rng.choice(["half", "interleaved"]),
                "norm": rng.random() < 0.75, "dtype": rng.choice(["bf16", "bf16", "fp32"]),
                "far": rng.choice([0, 1000, 1000000]), "factor": rng.choice([1.0, 8.0])}
    return {"op": "clip", "layers": _spread(rng, 1, 8), "d": _spread(rng, 64, 4096), "h": _spread(rng, 128, 11008),
            "mixed": rng.random() < 0.5, "clips": rng.random() < 0.75}


# ---- inputs ----

def _inv_freq(rot, factor):
    """Rotation frequencies 10000^(-2i/rot); for contexts `factor` times longer the slow ones are
    divided by it, the fast ones kept and those between blended (by turns over 4096 positions)."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    turns = 4096.0 * f / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    f = f * keep + f / factor * (1.0 - keep)
    return f.astype(np.float32), 1.0 if factor == 1.0 else 0.1 * math.log(factor) + 1.0


def _normal(gen, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32) * std).to(dtype)


def _weight(gen, n_in, n_out, layout):
    return _normal(gen, (n_in, n_out) if layout == "kn" else (n_out, n_in), n_in ** -0.5)


def _prepare_ffn(c, gen):
    M, d, h = c["M"], c["d"], c["h"]
    s = {"X": _normal(gen, (M, d)), "Wg": _weight(gen, d, h, c["layout"]), "Wu": _weight(gen, d, h, c["layout"]),
         "Wd": _weight(gen, h, d, c["layout"])}
    backward = c["op"] == "ffn_bwd"
    if backward:
        s["G"], s["U"] = _normal(gen, (M, h)), _normal(gen, (M, h))
        s["dY"] = _normal(gen, (M, d), 0.02)
    elif c["residual"]:
        s["R"] = _normal(gen, (M, d))
    if own:
        from gemm_epilogue_transformer_tiled_amd import block
        out = lambda like: torch.empty_like(like)  # noqa: E731
        s["plan"] = block.GatedFFN(M, d, h, act=c["act"], w_layout=c["layout"],
                                   residual=not backward and c["residual"], save=backward or c["save"])
        if backward:
            s["out"] = {"dX": out(s["X"]), "dWg": out(s["Wg"]), "dWu": out(s["Wu"]), "dWd": out(s["Wd"])}
            s["args"] = block.make_ffn_args(X=s["X"], Wg=s["Wg"], Wu=s["Wu"], Wd=s["Wd"], G=s["G"], U=s["U"],
                                            dY=s["dY"], **s["out"])
        else:
            s["out"] = {"Y": out(s["X"])}
            if c["save"]:
                s["out"].update(G=s["X"].new_empty(M, h), U=s["X"].new_empty(M, h))
            s["args"] = block.make_ffn_args(X=s["X"], Wg=s["Wg"], Wu=s["Wu"], Wd=s["Wd"], residual=s.get("R"),
                                            **s["out"])
    return s


def _prepare_qk(c, gen):
    T, hq, hk, D, rot = c["T"], c["hq"], c["hk"], c["D"], c["rot"]
    dtype = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    # queries, keys and values of a token lie side by side, as one projection writes them
    qkv = _normal(gen, (T, (hq + 2 * hk) * D), 1.0, dtype)
    q, k = qkv[:, :hq * D].view(T, hq, D), qkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
    if T <= 64:      # tokens of different sequences, each at its own position
        pos = torch.randint(0, c["far"] + 4096, (T,), generator=gen, device=DEVICE)
    else:            # two sequences, one after the other
        pos = torch.arange(T, device=DEVICE)
        pos = torch.where(pos < T // 3, pos, pos - T // 3) + c["far"]
    inv, amplitude = _inv_freq(rot, c["factor"])
    s = {"qkv": qkv, "q": q, "k": k, "pos": pos, "inv": torch.from_numpy(inv).to(DEVICE), "amplitude": amplitude,
         "gq": None, "gk": None}
    if c["norm"]:
        s["gq"] = (1 + 0.1 * torch.randn(D, generator=gen, device=DEVICE)).to(dtype)
        s["gk"] = (1 + 0.1 * torch.randn(D, generator=gen, device=DEVICE)).to(dtype)
    backward = c["op"] == "qk_bwd"
    if backward:
        s["doq"], s["dok"] = _normal(gen, (T, hq, D), 0.02, dtype), _normal(gen, (T, hk, D), 0.02, dtype)
    if own:
        from gemm_epilogue_transformer_tiled_amd import block
        s["plan"] = block.QKRotary(T, hq, hk, D, rot_dim=rot, pairs=c["pairs"], norm=c["norm"], eps=NORM_EPS,
                                   dtype=dtype, q_strides=q.stride()[:2], k_strides=k.stride()[:2])
        if backward:
            dqkv = torch.empty_like(qkv)
            dq, dk = dqkv[:, :hq * D].view(T, hq, D), dqkv[:, hq * D:(hq + hk) * D].view(T, hk, D)
            s["out"] = {"dq": dq, "dk": dk}
            if c["norm"]:
                s["out"].update(dgain_q=torch.empty(D, device=DEVICE), dgain_k=torch.empty(D, device=DEVICE))
            s["args"] = block.make_qk_args(q=q, k=k, positions=pos, inv_freq=s["inv"], amplitude=amplitude,
                                           gain_q=s["gq"], gain_k=s["gk"], dq_out=s["doq"], dk_out=s["dok"],
                                           **s["out"])
        else:
            s["out"] = {"q": torch.empty(T, hq, D, dtype=dtype, device=DEVICE),
                        "k": torch.empty(T, hk, D, dtype=dtype, device=DEVICE)}
            s["args"] = block.make_qk_args(q=q, k=k, q_out=s["out"]["q"], k_out=s["out"]["k"], positions=pos,
                                           inv_freq=s["inv"], amplitude=amplitude, gain_q=s["gq"], gain_k=s["gk"])
    return s


def _clip_shapes(c):
    """(shape, is a vector) of every gradient: a layer's three matrices, its gain and an odd vector."""
    d, h = c["d"], c["h"]
    return [((d, h), False), ((d, h), False), ((h, d), False), ((d,), True), ((h + 3,), True)] * c["layers"]


def _split(flat, shapes):
    got, at = [], 0
    for shape in shapes:
        n = math.prod(shape)
        got.append(flat[at:at + n].view(shape))
        at += n
    return got


def _prepare_clip(c, gen):
    shapes = _clip_shapes(c)
    big = [s for s, vector in shapes if not (c["mixed"] and vector)]
    small = [s for s, vector in shapes if c["mixed"] and vector]
    n = sum(math.prod(s) for s in big)
    # gradients of one parameter type lie in one buffer; max_norm 1 is exceeded, or far away
    std = (3.0 if c["clips"] else 0.05) * n ** -0.5
    flats = {"bf16": _normal(gen, (n,), std)}
    if small:
        flats["fp32"] = _normal(gen, (sum(math.prod(s) for s in small),), std, torch.float32)
    s = {"flats": flats, "grads": _split(flats["bf16"], big) + (_split(flats["fp32"], small) if small else []),
         "max_norm": 1.0}
    if own:
        from gemm_epilogue_transformer_tiled_amd import block
        clipped = {k: torch.empty_like(v) for k, v in flats.items()}
        outs = _split(clipped["bf16"], big) + (_split(clipped["fp32"], small) if small else [])
        s["out"] = {"norm": torch.empty(1, device=DEVICE), **clipped}
        s["plan"] = block.GradClip(s["grads"])
        s["args"] = block.make_clip_args(s["grads"], outs, norm=s["out"]["norm"], max_norm=s["max_norm"], eps=CLIP_EPS)
    return s


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(seed)
    op = case["op"]
    s = (_prepare_ffn if op.startswith("ffn") else _prepare_qk if op.startswith("qk") else _prepare_clip)(case, gen)
    s["case"] = case
    return s


# ---- plain forms ----

def _act(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    if name == "relu":
        return g * (g > 0)
    u = 0.7978845608028654 * (g + 0.044715 * g * g * g)
    return g / (1 + torch.exp(-2 * u))


def _act_grad(name, g):
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    if name == "relu":
        return (g > 0).float()
    s = 1 / (1 + torch.exp(-2 * 0.7978845608028654 * (g + 0.044715 * g * g * g)))
    return s + 2 * 0.7978845608028654 * g * s * (1 - s) * (1 + 3 * 0.044715 * g * g)


def _mat(s, name):
    """A weight as [in][out] in 32 bits."""
    w = s[name].float()
    return w if s["case"]["layout"] == "kn" else w.t()


def _plain_ffn_fwd(s):
    c, x = s["case"], s["X"].float()
    g, u = x @ _mat(s, "Wg"), x @ _mat(s, "Wu")
    y = (_act(c["act"], g) * u) @ _mat(s, "Wd")
    if "R" in s:
        y = y + s["R"].float()
    out = {"Y": y.bfloat16()}
    if c["save"]:
        out.update(G=g.bfloat16(), U=u.bfloat16())
    return out


def _plain_ffn_bwd(s):
    c, x, g, u, dy = s["case"], s["X"].float(), s["G"].float(), s["U"].float(), s["dY"].float()
    a = _act(c["act"], g)
    dh = dy @ _mat(s, "Wd").t()
    dg, du = dh * u * _act_grad(c["act"], g), dh * a
    back = (lambda w: w) if c["layout"] == "kn" else (lambda w: w.t().contiguous())
    return {"dX": (dg @ _mat(s, "Wg").t() + du @ _mat(s, "Wu").t()).bfloat16(),
            "dWg": back((x.t() @ dg).bfloat16()), "dWu": back((x.t() @ du).bfloat16()),
            "dWd": back(((a * u).t() @ dy).bfloat16())}


def _angles(s):
    """cos and sin, times the amplitude, of every token's rotation angles: [T][1][rot / 2]."""
    a = (s["pos"].double()[:, None] * s["inv"].double()[None, :])[:, None, :]
    return (torch.cos(a) * s["amplitude"]).float(), (torch.sin(a) * s["amplitude"]).float()


def _turn(x, cos, sin, c):
    """The first `rot` values of every head turned in pairs; the others as they are."""
    rot = c["rot"]
    if c["pairs"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_qk_fwd(s):
    c, (cos, sin) = s["case"], _angles(s)

    def one(x, gain):
        y = x.float()
        if gain is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + NORM_EPS) * gain.float()
        return _turn(y, cos, sin, c).to(x.dtype)
    return {"q": one(s["q"], s["gq"]), "k": one(s["k"], s["gk"])}


def _plain_qk_bwd(s):
    c, (cos, sin) = s["case"], _angles(s)

    def one(x, gain, dout):
        dy = _turn(dout.float(), cos, -sin, c)
        if gain is None:
            return dy.to(x.dtype), None
        xf = x.float()
        r = 1 / torch.sqrt((xf * xf).mean(-1, keepdim=True) + NORM_EPS)
        n = xf * r
        dn = dy * gain.float()
        dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        return dx.to(x.dtype), (dy.double() * n.double()).sum((0, 1)).float()
    dq, dgq = one(s["q"], s["gq"], s["doq"])
    dk, dgk = one(s["k"], s["gk"], s["dok"])
    out = {"dq": dq, "dk": dk}
    if c["norm"]:
        out.update(dgain_q=dgq, dgain_k=dgk)
    return out


def _plain_clip(s):
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
    norm = torch.sqrt(total).float()
    coef = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
    return {"norm": norm.reshape(1), **{k: (v.float() * coef).to(v.dtype) for k, v in s["flats"].items()}}


def run(s):
    op = s["case"]["op"]
    if own:
        if op == "ffn_fwd":
            s["plan"].forward(s["args"])
        elif op == "ffn_bwd":
            s["plan"].backward(s["args"])
        elif op == "qk_fwd":
            s["plan"].forward(s["args"])
        elif op == "qk_bwd":
            s["plan"].backward(s["args"])
        else:
            s["plan"].run(s["args"])
        return s["out"]
    return {"ffn_fwd": _plain_ffn_fwd, "ffn_bwd": _plain_ffn_bwd, "qk_fwd": _plain_qk_fwd, "qk_bwd": _plain_qk_bwd,
            "clip": _plain_clip}[op](s)


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op.startswith("ffn"):
        kn = case["layout"] == "kn"
        w = {k: s[k].to(f64) if kn else s[k].to(f64).t() for k in ("Wg", "Wu", "Wd")}
        act = {"silu": lambda t: t * torch.special.expit(t), "relu": lambda t: t.clamp(min=0),
               "gelu_tanh": lambda t: 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))}
        f, X = act[case["act"]], s["X"].to(f64)
        if op == "ffn_fwd":
            G, U = X @ w["Wg"], X @ w["Wu"]
            Y = (f(G) * U) @ w["Wd"]
            if case["residual"]:
                Y += s["R"].to(f64)
            return {"Y": Y, **({"G": G, "U": U} if case["save"] else {})}
        G = s["G"].to(f64).requires_grad_(True)
        with torch.enable_grad():
            A = f(G)
            slope, = torch.autograd.grad(A.sum(), G)
        A, U, dY = A.detach(), s["U"].to(f64), s["dY"].to(f64)
        dWd = (A * U).T @ dY
        dH = dY @ w["Wd"].T
        dU, dG = dH * A, dH * U * slope
        d = {"dX": dG @ w["Wg"].T + dU @ w["Wu"].T, "dWg": X.T @ dG, "dWu": X.T @ dU, "dWd": dWd}
        return {k: v if kn or k == "dX" else v.T.contiguous() for k, v in d.items()}
    if op.startswith("qk"):
        rot, D = case["rot"], case["D"]
        angle = torch.outer(s["pos"].to(f64), s["inv"].to(f64))
        turn = torch.polar(torch.full_like(angle, s["amplitude"]), angle)[:, None, :]     # a + ib -> (a + ib) e^(i angle)
        first = torch.arange(0, rot // 2, device=DEVICE) if case["pairs"] == "half" else torch.arange(0, rot, 2, device=DEVICE)
        second = first + (rot // 2 if case["pairs"] == "half" else 1)

        def rotate(x, by):
            z = torch.complex(x[..., first], x[..., second]) * by
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y
        out = {}
        for name, x, gain, dout in (("q", s["q"], s["gq"], s.get("doq")), ("k", s["k"], s["gk"], s.get("dok"))):
            x = x.to(f64)
            inv = (x.pow(2).sum(-1, keepdim=True) / D + NORM_EPS).rsqrt() if gain is not None else None
            g = gain.to(f64) if gain is not None else 1.0
            if op == "qk_fwd":
                out[name] = rotate(x * inv * g if gain is not None else x, turn)
                continue
            dy = rotate(dout.to(f64), turn.conj())
            if gain is None:
                out["d" + name] = dy
                continue
            along = (dy * g * x).sum(-1, keepdim=True) / D
            out["d" + name] = dy * g * inv - x * along * inv ** 3
            out["dgain_" + name] = (dy * x * inv).sum(0).sum(0)
        return out
    norm = math.sqrt(sum(float(v.to(f64).pow(2).sum()) for v in s["flats"].values()))
    coef = min(1.0, s["max_norm"] / (norm + CLIP_EPS))
    return {"norm": torch.tensor([norm], dtype=f64), **{k: v.to(f64) * coef for k, v in s["flats"].items()}}


def work(case):
    op = case["op"]
    if op.startswith("ffn"):
        M, d, h = case["M"], case["d"], case["h"]
        if op == "ffn_fwd":
            # X, three weights and R read, Y (and the kept G, U) written; three products
            values = 2 * M * d + 3 * d * h + (M * d if case["residual"] else 0) + (2 * M * h if case["save"] else 0)
            return {"bytes": 2 * values, "flops": 6 * M * d * h}
        # X, dY, G, U and the weights read, dX and the weights' gradients written; six products
        return {"bytes": 2 * (3 * M * d + 2 * M * h + 6 * d * h), "flops": 12 * M * d * h}
    if op.startswith("qk"):
        size = 2 if case["dtype"] == "bf16" else 4
        values = case["T"] * (case["hq"] + case["hk"]) * case["D"]
        back = op == "qk_bwd"
        # forward: queries and keys read and written; backward: dout and (with the norm) the inputs read
        return {"bytes": size * values * (3 if back and case["norm"] else 2) + 8 * case["T"],
                "flops": values * (20 if back else 10)}
    bf16 = sum(math.prod(s) for s, vector in _clip_shapes(case) if not (case["mixed"] and vector))
    fp32 = sum(math.prod(s) for s, vector in _clip_shapes(case) if case["mixed"] and vector)
    # every gradient read once, every clipped one written once
    return {"bytes": 2 * (2 * bf16 + 4 * fp32), "flops": 3 * (bf16 + fp32)}

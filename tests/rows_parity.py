"""64-bit references of the row operators and elementwise bounds on what the kernels may be off by,
derived from the roundings they make.

u (half_step) bounds one rounding to the element type relative to the value: 2^-8 bf16, 2^-24 fp32; e = 2^-24
one fp32 operation.  A sum of D values in fp32, in any order, is off by at most D e sum|v| (to first order;
D + 8 covers the second)."""
from __future__ import annotations

import numpy as np
import torch

from tests.block_parity import E, F, TINY, act, check, half_step  # noqa: F401

STEPS = 65536


def _mulhilo(a, m):
    p = a.astype(np.uint64) * np.uint64(m)
    return (p >> np.uint64(32)).astype(np.uint32), p.astype(np.uint32)


def philox(counter, key):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) of uint32 arrays: four counter words, two key words."""
    c, (k0, k1) = [np.asarray(w, np.uint32) for w in counter], (int(k) for k in key)
    for _ in range(10):
        h0, l0 = _mulhilo(c[0], 0xD2511F53)
        h1, l1 = _mulhilo(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ np.uint32(k0), l1, h0 ^ c[3] ^ np.uint32(k1), l0]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def drop_factors(rows, d, p, seed, offset, site):
    """What each value is multiplied with: 0 where it is dropped."""
    t = int(np.floor(float(np.float32(p)) * STEPS + 0.5))
    nb = -(-d // 8)
    n = rows * nb
    full = lambda v: np.full(n, v & 0xFFFFFFFF, np.uint32)  # noqa: E731
    w = philox((np.arange(n, dtype=np.uint32), full(site), full(offset), full(offset >> 32)),
               (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF))
    half = np.stack([h for x in w for h in (x & np.uint32(0xFFFF), x >> np.uint32(16))], -1).reshape(rows, nb * 8)[:, :d]
    return torch.from_numpy((half >= t) * (STEPS / (STEPS - t)))


def drop(x, factors):
    """x times its factors; a dropped value is 0 whatever it was."""
    return x if factors is None else torch.where(factors == 0, torch.zeros((), dtype=x.dtype, device=x.device), x * factors)


def norm_sum(X, R, factors):
    """(s, bound): the sum in front of the norm in 64 bits and the bound on the kept one."""
    x = drop(X.double(), factors)
    s = x if R is None else R.double() + x
    off = 0.0 if factors is None and R is None else 4 * E * (x.abs() + s.abs())
    return s, half_step(X.dtype) * s.abs() * (R is not None or factors is not None) + (1 + half_step(X.dtype)) * off + TINY


def norm_forward(S, gain, bias, eps):
    """{Y, mean, rstd} of the kept sum S and their bounds."""
    s, half, D = S.double(), half_step(S.dtype), S.shape[1]
    k = (D + 8) * E
    mean = s.mean(1, keepdim=True)
    tmean = k * s.abs().mean(1, keepdim=True) + E * mean.abs()
    c = s - mean
    var = (c * c).mean(1, keepdim=True)
    # each c is off by tmean (the same for all: to first order their sum cancels, to second it is its square)
    # and its own rounding
    own = E * (s.abs() + tmean)
    tvar = k * var + tmean ** 2 + 2 * (c.abs() * own).mean(1, keepdim=True) + (own ** 2).mean(1, keepdim=True) \
        + 2 * tmean * own.mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    tr = r * (0.5 * tvar / (var + eps) * 1.01 + 4 * E)
    g = gain.double() if gain is not None else torch.ones(D, dtype=torch.float64, device=S.device)
    b = bias.double() if bias is not None else torch.zeros(D, dtype=torch.float64, device=S.device)
    y = c * r * g + b
    ty = g.abs() * ((tmean + own) * (r + tr) + c.abs() * tr + 2 * E * (c.abs() + tmean) * r) + E * (y.abs() + (c * r * g).abs())
    ref = {"Y": y, "mean": mean[:, 0], "rstd": r[:, 0]}
    tol = {"Y": half * y.abs() + (1 + half) * ty + TINY, "mean": tmean[:, 0] + TINY, "rstd": tr[:, 0] + TINY}
    return ref, tol


def norm_backward(dY, S, dS, mean, rstd, gain, factors):
    """{dX, dR, dgain, dbias} in 64 bits and their bounds (mean and rstd as given)."""
    half, (M, D) = half_step(S.dtype), S.shape
    k = (D + 8) * E
    dy, r = dY.double(), rstd.double()[:, None]
    n = (S.double() - mean.double()[:, None]) * r
    tn = E * (n.abs() + (S.double() - mean.double()[:, None]).abs() * r)
    g = gain.double() if gain is not None else torch.ones(D, dtype=torch.float64, device=S.device)
    e = dy * g
    te = E * e.abs()
    me, men = e.mean(1, keepdim=True), (e * n).mean(1, keepdim=True)
    tme = k * e.abs().mean(1, keepdim=True) + te.mean(1, keepdim=True) + E * me.abs()
    tmen = k * (e * n).abs().mean(1, keepdim=True) + (te * n.abs() + e.abs() * tn).mean(1, keepdim=True) + E * men.abs()
    inner = e - me - n * men
    ti = te + tme + tn * men.abs() + n.abs() * tmen + 2 * E * (e.abs() + me.abs() + (n * men).abs())
    out, tout = r * inner, r * (ti + E * inner.abs())
    if dS is not None:
        out, tout = out + dS.double(), tout + E * (out.abs() + dS.double().abs())
    dx = drop(out, factors)
    big = 1.0 if factors is None else float(factors.max())
    tdx = big * (tout + 2 * E * out.abs())
    if factors is not None:
        tdx = torch.where(factors == 0, torch.zeros_like(tdx), tdx)
    ks = (M + 16) * E
    dg, db = (dy * n).sum(0), dy.sum(0)
    ref = {"dX": dx, "dR": out, "dgain": dg, "dbias": db}
    tol = {"dX": half * dx.abs() + (1 + half) * tdx + TINY, "dR": half * out.abs() + (1 + half) * tout + TINY,
           "dgain": (ks * (dy * n).abs() + dy.abs() * tn).sum(0) + E * dg.abs() + TINY,
           "dbias": (ks * dy.abs()).sum(0) + E * db.abs() + TINY}
    return ref, tol


def quant(X):
    """(codes, scale) by the definition, in 64 bits (the quotient of 32-bit values is exact enough to decide
    every tie: any other quotient is 2^-33 away from one)."""
    x = X.double()
    if x.shape[1] == 0:
        return torch.zeros(x.shape, dtype=torch.int8, device=x.device), torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    a = x.abs().amax(1)
    sound = torch.isfinite(x).all(1)
    q = 127 * x / torch.where(a > 0, a, torch.ones_like(a))[:, None]
    codes = torch.where(sound[:, None], torch.round(torch.where(sound[:, None], q, torch.zeros_like(q))), torch.zeros_like(q))
    return codes.to(torch.int8), torch.where(sound, a / 127, torch.full_like(a, float("nan")))


def int8(X, W, x_scale, w_scale, bias, R, name, dtype):
    """(Y, bound).  The sum is exact; its conversion, the two scales and the bias round in fp32; the activation is
    within F (1 + |t|) of its value (block_parity) and its slope below 1.13."""
    half = half_step(dtype)
    raw = (X.double() @ W.double().t()) * x_scale.double()[:, None] * w_scale.double()
    t = raw if bias is None else raw + bias.double()
    tt = 4 * E * raw.abs() + E * t.abs()
    y = act(name, t)
    ty = 1.13 * tt + (F * (1 + t.abs()) if name in ("silu", "gelu_tanh") else 0.0)
    if R is not None:
        y = y + R.double()
        ty = ty + E * y.abs()
    return y, half * y.abs() + (1 + half) * ty + TINY

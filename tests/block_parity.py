"""64-bit references of the transformer-block operators and elementwise bounds on what the kernels
may be off by, derived from the roundings they make.

u = 2^-8 bounds one rounding to bf16 relative to the value, e = 2^-24 one fp32 operation.  A sum of
K products in fp32, in any order, is off by at most K e sum|a||b| (to first order; K + 8 covers the
second).  The activations use the hardware's exp2 and reciprocal, each within 2^-22 relative: an
activation of g is within 2^-19 (1 + |g|) |act bound|, which F below carries."""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8
E = 2.0 ** -24
F = 2.0 ** -19
TINY = 2.0 ** -126


def act(name, g):
    if name == "none":
        return g
    if name == "relu":
        return g.clamp(min=0)
    if name == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def act_grad(name, g):
    if name == "none":
        return torch.ones_like(g)
    if name == "relu":
        return (g > 0).to(g.dtype)
    if name == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _mat(w, layout):
    w = w.double()
    return w if layout == "kn" else w.t()


def ffn_forward(X, Wg, Wu, Wd, name, layout, R=None):
    """{"Y", "G", "U"} in 64 bits and the bound on each."""
    x, wg, wu, wd = X.double(), _mat(Wg, layout), _mat(Wu, layout), _mat(Wd, layout)
    d, h = wg.shape
    g, u = x @ wg, x @ wu
    ag, au = (d + 8) * E * (x.abs() @ wg.abs()), (d + 8) * E * (x.abs() @ wu.abs())
    a = act(name, g)
    hid = a * u
    # every activation's slope is below 1.13 in size
    th = U * hid.abs() + (1.13 * ag + F * (1 + g.abs())) * (u.abs() + au) + (a.abs() + 1.13 * ag) * au
    y = hid @ wd
    ty = (1 + U) * th @ wd.abs() + (h + 8) * E * ((hid.abs() + th) @ wd.abs())
    if R is not None:
        y = y + R.double()
        ty = ty + E * y.abs()
    ref = {"Y": y, "G": g, "U": u}
    tol = {"Y": ty + U * (y.abs() + ty) + TINY, "G": ag + U * (g.abs() + ag) + TINY, "U": au + U * (u.abs() + au) + TINY}
    return ref, tol


def ffn_backward(X, Wg, Wu, Wd, G, Uv, dY, name, layout):
    """{"dX", "dWg", "dWu", "dWd"} in 64 bits and the bound on each."""
    x, wg, wu, wd = X.double(), _mat(Wg, layout), _mat(Wu, layout), _mat(Wd, layout)
    g, u, dy = G.double(), Uv.double(), dY.double()
    d, h = wg.shape
    M = x.shape[0]
    a, s = act(name, g), act_grad(name, g)
    dh = dy @ wd.t()
    adh = (d + 8) * E * (dy.abs() @ wd.t().abs())
    ta = F * (1 + g.abs()) if name != "none" else torch.zeros_like(g)
    dg, du, hid = dh * u * s, dh * a, a * u
    big = dh.abs() + adh
    tg = U * dg.abs() + (1 + U) * u.abs() * (1.13 * adh + big * (ta + 4 * E))
    tu = U * du.abs() + (1 + U) * (a.abs() * adh + big * (ta + 4 * E))
    th = U * hid.abs() + (1 + U) * u.abs() * (ta + 4 * E)

    def product(p, tp, q, k):
        """p @ q with p off by tp, summed over k in fp32, rounded once to bf16: value and bound."""
        v = p @ q
        t = tp @ q.abs() + (k + 8) * E * ((p.abs() + tp) @ q.abs())
        return v, t

    d1, t1 = product(dg, tg, wg.t(), 2 * h)
    d2, t2 = product(du, tu, wu.t(), 2 * h)
    pairs = {"dX": (d1 + d2, t1 + t2)}
    for n, left, tl in (("dWg", dg, tg), ("dWu", du, tu)):
        v, t = product(left.t(), tl.t(), x, M)          # (X^T dG)^T
        pairs[n] = (v.t(), t.t())
    pairs["dWd"] = product(hid.t(), th.t(), dy, M)
    ref = {k: v for k, (v, t) in pairs.items()}
    tol = {k: t + U * (v.abs() + t) + TINY for k, (v, t) in pairs.items()}
    if layout == "nk":
        for k in ("dWg", "dWu", "dWd"):
            ref[k], tol[k] = ref[k].t(), tol[k].t()
    return ref, tol


def check(got, ref, tol, what):
    """Every element of got within tol of ref."""
    off = (got.double() - ref).abs()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(off <= tol)
    if bad.any():
        i = int(torch.nan_to_num(off / tol, nan=math.inf).flatten().argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: got "
                             f"{float(got.double().flatten()[i])}, want {float(ref.flatten()[i])} +- {float(tol.flatten()[i])}")

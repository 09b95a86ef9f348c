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


# ---- query/key norm with rotation ----
# The angle is reduced to a turn in 64 bits and rounded once to fp32 (2^-25 of a turn, 2^-22.3 rad); its
# cosine and sine add two units of 2^-24: ANGLE bounds the error of either.
ANGLE = 2.0 ** -21


def _turned(a, b, cos, sin):
    return a * cos - b * sin, b * cos + a * sin


def qk(x, dout, gain, pos, inv, amplitude, rot, pairs, eps):
    """64-bit (out, tol) of one of queries or keys, or with dout (dx, tol, dgain, tol of dgain)."""
    T, H, D = x.shape
    x, half = x.double(), U if x.dtype == torch.bfloat16 else E
    first = torch.arange(rot // 2, device=x.device) if pairs == "half" else torch.arange(0, rot, 2, device=x.device)
    second = first + (rot // 2 if pairs == "half" else 1)
    angle = pos.double()[:, None] * inv.double()[None, :]
    cos, sin = amplitude * torch.cos(angle)[:, None], amplitude * torch.sin(angle)[:, None]
    steps = (D + 16) * E

    def rotate(v, s):
        y = v.clone()
        y[..., first], y[..., second] = _turned(v[..., first], v[..., second], cos, s)
        size = v.abs()
        both = abs(amplitude) * (v[..., first].abs() + v[..., second].abs())
        size[..., first], size[..., second] = both, both
        return y, size
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if gain is not None else None
    if dout is None:
        y = x * r * gain.double() if gain is not None else x
        out, size = rotate(y, sin)
        return out, half * out.abs() + (1 + half) * size * (ANGLE + steps) + TINY
    dy, size = rotate(dout.double(), -sin)
    tdy = size * (ANGLE + 4 * E)
    if gain is None:
        return dy, half * dy.abs() + (1 + half) * tdy + TINY, None, None
    n, g = x * r, gain.double()
    e, te = dy * g, tdy * g.abs() + steps * (dy * g).abs()
    mean = (e * n).mean(-1, keepdim=True)
    tmean = (te * n.abs()).mean(-1, keepdim=True) + steps * (e * n).abs().mean(-1, keepdim=True)
    dx = r * (e - n * mean)
    tdx = r * (te + n.abs() * tmean + 2 * steps * (e.abs() + (n * mean).abs()))
    dgain = (dy * n).sum((0, 1))
    tgain = (tdy * n.abs() + (steps + (T * H + 16) * E) * (dy * n).abs()).sum((0, 1))
    return dx, half * dx.abs() + (1 + half) * tdx + TINY, dgain, tgain + E * dgain.abs() + TINY


def half_step(dtype):
    return U if dtype == torch.bfloat16 else E

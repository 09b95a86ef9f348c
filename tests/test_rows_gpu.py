"""The row operators on the GPU against their 64-bit definitions: layer norm with dropout and residual, forward
and backward, dropout, int8 codes and the product of codes, at the sizes, layouts and values where they can
go wrong."""
from __future__ import annotations

import math

import pytest
import torch

from tests import rows_parity as rp

pytestmark = pytest.mark.gpu

rows = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.rows")

BF16, FP32 = torch.bfloat16, torch.float32
SEED, OFFSET, SITE = 0x1234567890ABCDEF, (5 << 32) + 77, 9


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def rng_of(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


def factors_of(M, d, p, site=SITE):
    return rp.drop_factors(M, d, p, SEED, OFFSET, site).cuda() if p else None


def normal(gen, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)


def padded(t, ld):
    """The same matrix with rows ld apart and a canary between them."""
    if t is None or ld is None:
        return t
    buf = torch.full((t.shape[0], ld), 77, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def canary_ok(view):
    ld, d = view.stride(0), view.shape[1]
    whole = view.as_strided((view.shape[0], ld), (ld, 1), view.storage_offset())
    return bool((whole[:, d:] == 77).all()) if view.shape[0] else True


# ---- layer norm ----

# every row shape and both its borders, odd widths, one value
WIDTHS = [1, 3, 7, 8, 9, 64, 65, 511, 512, 520, 1021, 1024, 1032, 2047, 2048, 2056, 4096, 4100, 8192, 8200, 16384, 16385, 32768]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_forward_widths(d, dtype):
    gen = torch.Generator("cuda").manual_seed(d)
    M = 5
    X, gain, bias = normal(gen, (M, d), dtype, 2.0, 0.5), normal(gen, (d,), dtype, 0.2, 1.0), normal(gen, (d,), dtype)
    Y, mean, rstd = torch.empty_like(X), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    plan = rows.LayerNorm(M, d, dtype=dtype)
    plan.forward(rows.make_norm_args(X=X, Y=Y, gain=gain, bias=bias, mean=mean, rstd=rstd))
    ref, tol = rp.norm_forward(X, gain, bias, 1e-5)
    for n, got in (("Y", Y), ("mean", mean), ("rstd", rstd)):
        rp.check(got, ref[n], tol[n], (n, d))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_backward_widths(d, dtype):
    gen = torch.Generator("cuda").manual_seed(d)
    M = 13
    S, dY, dS, gain = (normal(gen, (M, d), dtype, 2.0, 0.5), normal(gen, (M, d), dtype, 0.05), normal(gen, (M, d), dtype, 0.05),
                       normal(gen, (d,), dtype, 0.2, 1.0))
    x = S.double()
    mean, rstd = x.mean(1).float(), (1 / torch.sqrt(x.var(1, correction=0) + 1e-5)).float()
    dX, dgain, dbias = torch.empty_like(S), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    plan = rows.LayerNorm(M, d, dtype=dtype)
    plan.backward(rows.make_norm_args(S=S, dY=dY, dS=dS, gain=gain, mean=mean, rstd=rstd, dX=dX, dgain=dgain, dbias=dbias))
    ref, tol = rp.norm_backward(dY, S, dS, mean, rstd, gain, None)
    for n, got in (("dX", dX), ("dgain", dgain), ("dbias", dbias)):
        rp.check(got, ref[n], tol[n], (n, d))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,d,pad", [(1, 1000, 0), (37, 1021, 0), (300, 264, 8), (19, 100, 3), (1500, 72, 0), (4100, 2304, 0)])
def test_norm_with_dropout_and_residual(M, d, pad, residual, p, dtype):
    gen = torch.Generator("cuda").manual_seed(M + d)
    ld = d + pad if pad else None
    lds = {n: d + pad for n in ("ldx", "ldr", "lds", "ldy", "lddy", "ldds", "lddx", "lddr")} if pad else {}
    X, R = padded(normal(gen, (M, d), dtype), ld), padded(normal(gen, (M, d), dtype, 2.0, 0.3), ld) if residual else None
    gain, bias = normal(gen, (d,), dtype, 0.2, 1.0), normal(gen, (d,), dtype)
    new = lambda: padded(torch.full((M, d), float("nan"), dtype=dtype, device="cuda"), ld)  # noqa: E731
    S, Y, mean, rstd = new(), new(), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    plan = rows.LayerNorm(M, d, dtype=dtype, residual=residual, dropout=p, site=SITE, **lds)
    rng = rng_of()
    plan.forward(rows.make_norm_args(X=X, residual=R, S=S, Y=Y, gain=gain, bias=bias, mean=mean, rstd=rstd, rng=rng))
    f = factors_of(M, d, p)
    s, ts = rp.norm_sum(X, R, f)
    rp.check(S, s, ts, "S")
    ref, tol = rp.norm_forward(S, gain, bias, 1e-5)
    for n, got in (("Y", Y), ("mean", mean), ("rstd", rstd)):
        rp.check(got, ref[n], tol[n], n)
    dY, dS = padded(normal(gen, (M, d), dtype, 0.05), ld), padded(normal(gen, (M, d), dtype, 0.05), ld)
    dX, dR, dgain, dbias = new(), new(), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    plan.backward(rows.make_norm_args(S=S, mean=mean, rstd=rstd, gain=gain, rng=rng, dY=dY, dS=dS, dX=dX, dR=dR, dgain=dgain,
                                      dbias=dbias))
    ref, tol = rp.norm_backward(dY, S, dS, mean, rstd, gain, f)
    for n, got in (("dX", dX), ("dR", dR), ("dgain", dgain), ("dbias", dbias)):
        rp.check(got, ref[n], tol[n], n)
    if p:
        assert bool((dX[f == 0] == 0).all())
    if pad:
        assert all(canary_ok(t) for t in (S, Y, dX, dR))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [8200, 11008, 16383, 16392, 32767, 32768])
def test_norm_backward_of_many_wide_rows(d, dtype):
    """Several rows a workgroup, with everything a call can have and over its inputs."""
    M = 600
    gen = torch.Generator("cuda").manual_seed(d)
    S, dY, dS, gain = (normal(gen, (M, d), dtype, 2.0, 0.5), normal(gen, (M, d), dtype, 0.05), normal(gen, (M, d), dtype, 0.05),
                       normal(gen, (d,), dtype, 0.2, 1.0))
    x = S.double()
    mean, rstd = x.mean(1).float(), (1 / torch.sqrt(x.var(1, correction=0) + 1e-5)).float()
    del x
    plan = rows.LayerNorm(M, d, dtype=dtype, residual=True, dropout=0.25, site=SITE)
    for g, add in ((gain, dS), (None, None)):
        f = factors_of(M, d, 0.25)
        ref, tol = rp.norm_backward(dY, S, add, mean, rstd, g, f)
        dX, dgain, dbias = dY.clone(), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
        dR = dS.clone() if add is not None else torch.empty_like(dY)
        plan.backward(rows.make_norm_args(S=S, mean=mean, rstd=rstd, gain=g, rng=rng_of(), dY=dX, dS=dR if add is not None else None,
                                          dX=dX, dR=dR, dgain=dgain, dbias=dbias))
        for n, got in (("dX", dX), ("dR", dR), ("dgain", dgain), ("dbias", dbias)):
            rp.check(got, ref[n], tol[n], (n, d))
        del f, ref, tol


def test_norm_optional_outputs_and_in_place():
    """Every subset of outputs gives the same bits; S over R, Y over X, dX over dY, dR over dS."""
    M, d = 70, 520
    gen = torch.Generator("cuda").manual_seed(1)
    X, R, gain, bias = (normal(gen, (M, d), BF16), normal(gen, (M, d), BF16), normal(gen, (d,), BF16, 0.2, 1.0),
                        normal(gen, (d,), BF16))
    plan = rows.LayerNorm(M, d, residual=True, dropout=0.2, site=3)
    rng = rng_of()
    e = lambda: torch.empty_like(X)  # noqa: E731
    S, Y, mean, rstd = e(), e(), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    common = dict(gain=gain, bias=bias, rng=rng)
    plan.forward(rows.make_norm_args(X=X, residual=R, S=S, Y=Y, mean=mean, rstd=rstd, **common))
    Y2 = e()
    plan.forward(rows.make_norm_args(X=X, residual=R, Y=Y2, **common))
    assert torch.equal(Y, Y2)
    x2, r2 = X.clone(), R.clone()
    plan.forward(rows.make_norm_args(X=x2, residual=r2, S=r2, Y=x2, **common))
    assert torch.equal(x2, Y) and torch.equal(r2, S)
    plain = e()
    plan.forward(rows.make_norm_args(X=X, residual=R, Y=plain, rng=rng))
    rp.check(plain, *[v["Y"] for v in rp.norm_forward(S, None, None, 1e-5)], "without gain and bias")
    dY, dS = normal(gen, (M, d), BF16, 0.1), normal(gen, (M, d), BF16, 0.1)
    v = lambda: torch.empty(d, device="cuda")  # noqa: E731
    dX, dR, dg, db = e(), e(), v(), v()
    back = dict(S=S, mean=mean, rstd=rstd, gain=gain, rng=rng)
    plan.backward(rows.make_norm_args(dY=dY, dS=dS, dX=dX, dR=dR, dgain=dg, dbias=db, **back))
    for kw in (dict(dX=e()), dict(dR=e()), dict(dgain=v()), dict(dbias=v()), dict(dX=e(), dbias=v())):
        plan.backward(rows.make_norm_args(dY=dY, dS=dS, **kw, **back))
        for n, got in kw.items():
            assert torch.equal(got, {"dX": dX, "dR": dR, "dgain": dg, "dbias": db}[n]), n
    a, b = dY.clone(), dS.clone()
    plan.backward(rows.make_norm_args(dY=a, dS=b, dX=a, dR=b, **back))
    assert torch.equal(a, dX) and torch.equal(b, dR)
    without = e()
    plan.backward(rows.make_norm_args(dY=dY, dR=without, S=S, mean=mean, rstd=rstd))
    ref, tol = rp.norm_backward(dY, S, None, mean, rstd, None, None)
    rp.check(without, ref["dR"], tol["dR"], "no gain, no dS")


def test_norm_of_no_rows():
    d = 40
    plan = rows.LayerNorm(0, d)
    e = torch.empty(0, d, dtype=BF16, device="cuda")
    plan.forward(rows.make_norm_args(X=e, Y=e.clone()))
    dg, db = torch.full((d,), 5.0, device="cuda"), torch.full((d,), 5.0, device="cuda")
    plan.backward(rows.make_norm_args(dY=e, S=e, mean=torch.empty(0, device="cuda"), rstd=torch.empty(0, device="cuda"),
                                      dX=e.clone(), dgain=dg, dbias=db))
    assert bool((dg == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("d", [24, 1000, 5000])
def test_norm_values(d):
    """Rows far from zero, of equal values, with infinities and NaN: neighbours are not touched."""
    gen = torch.Generator("cuda").manual_seed(d)
    X = normal(gen, (7, d), FP32)
    X[1] += 1000.0
    X[2] = 3.5
    X[3, d // 2] = math.inf
    X[4, d - 1] = math.nan
    X[5] *= 1e-3
    gain, bias = normal(gen, (d,), FP32, 0.2, 1.0), normal(gen, (d,), FP32)
    Y, mean, rstd = torch.empty_like(X), torch.empty(7, device="cuda"), torch.empty(7, device="cuda")
    rows.LayerNorm(7, d, dtype=FP32).forward(rows.make_norm_args(X=X, Y=Y, gain=gain, bias=bias, mean=mean, rstd=rstd))
    good = [0, 1, 2, 5, 6]
    ref, tol = rp.norm_forward(X[good], gain, bias, 1e-5)
    rp.check(Y[good], ref["Y"], tol["Y"], "Y")
    rp.check(rstd[good], ref["rstd"], tol["rstd"], "rstd")
    assert torch.equal(Y[2], bias)
    assert bool(Y[[3, 4]].isnan().all())


def test_norm_gradient_against_differences():
    """The gradients of f = sum(W * Y) + sum(V * S) by central differences in 64 bits of the definition."""
    M, d, p = 4, 23, 0.25
    gen = torch.Generator("cuda").manual_seed(5)
    X, R, gain, bias = (normal(gen, (M, d), FP32), normal(gen, (M, d), FP32), normal(gen, (d,), FP32, 0.2, 1.0),
                        normal(gen, (d,), FP32))
    W, V = normal(gen, (M, d), FP32), normal(gen, (M, d), FP32)
    f = factors_of(M, d, p)

    def value(x, r, g, b):
        s = r + x * f
        c = s - s.mean(1, keepdim=True)
        y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * g + b
        return float((W.double() * y).sum() + (V.double() * s).sum())
    plan = rows.LayerNorm(M, d, dtype=FP32, residual=True, dropout=p, site=SITE)
    rng = rng_of()
    S, Y, mean, rstd = torch.empty_like(X), torch.empty_like(X), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    plan.forward(rows.make_norm_args(X=X, residual=R, S=S, Y=Y, gain=gain, bias=bias, mean=mean, rstd=rstd, rng=rng))
    dX, dR, dg, db = torch.empty_like(X), torch.empty_like(X), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    plan.backward(rows.make_norm_args(S=S, mean=mean, rstd=rstd, gain=gain, rng=rng, dY=W, dS=V, dX=dX, dR=dR, dgain=dg, dbias=db))
    at = [t.double() for t in (X, R, gain, bias)]
    h = 1e-5
    for which, got in enumerate((dX, dR, dg, db)):
        for i in range(0, got.numel(), 7):
            lo, hi = [t.clone() for t in at], [t.clone() for t in at]
            lo[which].view(-1)[i] -= h
            hi[which].view(-1)[i] += h
            slope = (value(*hi) - value(*lo)) / (2 * h)
            # the differences' own error: h^2 of third derivatives of order 10, 1e-16 of a value of 100 over h
            assert abs(float(got.view(-1)[i]) - slope) <= 1e-4 * (1 + abs(slope)), (which, i)


# ---- dropout ----

@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,d,pad", [(1, 1, 0), (3, 7, 0), (1, 8, 0), (5, 9, 4), (777, 1021, 0), (64, 1024, 0), (64, 1024, 8),
                                     (100, 96, 3), (3001, 2048, 0)])
def test_dropout(M, d, pad, residual, dtype):
    gen = torch.Generator("cuda").manual_seed(M * d)
    ld = d + pad if pad else None
    lds = {n: d + pad for n in ("ldx", "ldr", "ldy", "lddy", "lddx")} if pad else {}
    X, dY = padded(normal(gen, (M, d), dtype), ld), padded(normal(gen, (M, d), dtype), ld)
    R = padded(normal(gen, (M, d), dtype), ld) if residual else None
    Y, dX = padded(torch.empty_like(X), ld), padded(torch.empty_like(X), ld)
    p, rng = 0.3, rng_of()
    plan = rows.Dropout(M, d, p, dtype=dtype, residual=residual, site=SITE, **lds)
    args = rows.make_dropout_args(X=X, residual=R, Y=Y, dY=dY, dX=dX, rng=rng)
    plan.forward(args)
    plan.backward(args)
    f = factors_of(M, d, p)
    half = rp.half_step(dtype)
    want = X.double() * f + (R.double() if residual else 0)
    rp.check(Y, want, half * want.abs() + 3 * rp.E * ((X.double() * f).abs() + want.abs()) + rp.TINY, "Y")
    want = dY.double() * f
    rp.check(dX, want, (half + 3 * rp.E) * want.abs() + rp.TINY, "dX")
    if pad:
        assert canary_ok(Y) and canary_ok(dX)


@pytest.mark.parametrize("p", [0.0, 1 / 65536, 0.5, 65535 / 65536])
def test_dropout_probabilities(p):
    """The share that is dropped, the ends of the range, and values that are not finite."""
    M, d = 512, 1024
    X = torch.ones(M, d, device="cuda")
    Y = torch.empty_like(X)
    plan = rows.Dropout(M, d, p, dtype=FP32, site=SITE)
    plan.forward(rows.make_dropout_args(X=X, Y=Y, rng=rng_of()))
    f = rp.drop_factors(M, d, p, SEED, OFFSET, SITE).cuda()
    assert torch.equal(Y, f.float())
    n, zeros = M * d, int((Y == 0).sum())
    assert abs(zeros - n * p) <= 6 * math.sqrt(n * p * (1 - p)) + 1
    X.fill_(math.nan)
    plan.forward(rows.make_dropout_args(X=X, Y=Y, rng=rng_of()))
    assert bool((Y[f == 0] == 0).all()) and bool(Y[f != 0].isnan().all())


def test_dropout_numbers_are_those_of_the_key():
    """Another seed, offset or site is another mask; all 64 bits of seed and offset count; in place."""
    M, d, p = 40, 512, 0.5
    X = torch.ones(M, d, device="cuda")

    def mask(seed, offset, site):
        y = X.clone()
        rows.Dropout(M, d, p, dtype=FP32, site=site).forward(rows.make_dropout_args(X=y, Y=y, rng=rng_of(seed, offset)))
        assert torch.equal(y.cpu().double(), rp.drop_factors(M, d, p, seed, offset, site))
        return y
    seen = [mask(s, o, t) for s, o, t in ((1, 0, 0), (1 + (1 << 32), 0, 0), (-1, 0, 0), (1, 1, 0), (1, 1 << 32, 0), (1, -1, 0),
                                          (1, 0, 1), (1, 0, 0xFFFFFFFF))]
    for i, a in enumerate(seen):
        for b in seen[:i]:
            assert not torch.equal(a, b)


def test_norm_drops_what_dropout_drops():
    M, d, p = 33, 1000, 0.4
    gen = torch.Generator("cuda").manual_seed(0)
    X, R = normal(gen, (M, d), FP32), normal(gen, (M, d), FP32)
    rng, Y, S, out = rng_of(), torch.empty_like(X), torch.empty_like(X), torch.empty_like(X)
    rows.Dropout(M, d, p, dtype=FP32, residual=True, site=4).forward(rows.make_dropout_args(X=X, residual=R, Y=Y, rng=rng))
    rows.LayerNorm(M, d, dtype=FP32, residual=True, dropout=p, site=4).forward(
        rows.make_norm_args(X=X, residual=R, S=S, Y=out, rng=rng))
    rp.check(S, Y.double(), 2 * rp.E * (Y.double().abs() + 2 * X.double().abs()), "the same sum")


# ---- int8 codes ----

@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [0, 1, 7] + WIDTHS[3:])
def test_quant_widths(d, dtype):
    gen = torch.Generator("cuda").manual_seed(d)
    M = 9
    X = normal(gen, (M, d), dtype, 3.0)
    codes, scale = torch.full((M, d), 99, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    rows.RowQuant(M, d, dtype=dtype).run(rows.make_quant_args(X=X, codes=codes, scale=scale))
    want, ws = rp.quant(X)
    assert torch.equal(codes, want)
    rp.check(scale, ws, rp.E * ws + 2.0 ** -149, "scale")


@pytest.mark.parametrize("M,d,ldx,ldq", [(700, 264, 272, 300), (700, 263, 264, 263), (5000, 100, 100, 112), (3, 4097, 4097, 4100)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_quant_layouts(M, d, ldx, ldq, dtype):
    gen = torch.Generator("cuda").manual_seed(d)
    X = padded(normal(gen, (M, d), dtype), ldx)
    codes, scale = padded(torch.zeros(M, d, dtype=torch.int8, device="cuda"), ldq), torch.empty(M, device="cuda")
    rows.RowQuant(M, d, dtype=dtype, ldx=ldx, ldq=ldq).run(rows.make_quant_args(X=X, codes=codes, scale=scale))
    assert torch.equal(codes, rp.quant(X)[0]) and canary_ok(codes)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_quant_ties(dtype):
    """Every quotient that a bf16 maximum and value can have (and for fp32 the values next to them), at scales
    from the subnormal to the largest values."""
    m = torch.arange(128, 256, dtype=torch.float64)
    X = torch.cat([m[:, None], torch.cat([m, m / 2, m / 4, m / 8, m / 64, m / 256])[None].expand(128, -1).clamp(max=1e9)], 1)
    X = torch.where(X.abs() > m[:, None], -X / 2, X).cuda()
    for shift in (-133 - 7, -126, -70, -61, -60, -20, 0, 60, 120):
        x = (X * 2.0 ** shift).to(dtype)
        if dtype == FP32:
            x = torch.cat([x, torch.nextafter(x, torch.zeros_like(x)), torch.nextafter(x, torch.full_like(x, 1e38))[:, 1:]], 1)
            x = torch.where(x.abs() > x[:, :1].abs(), x[:, :1], x)
        codes, scale = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(128, device="cuda")
        rows.RowQuant(*x.shape, dtype=dtype).run(rows.make_quant_args(X=x, codes=codes, scale=scale))
        want, ws = rp.quant(x)
        assert torch.equal(codes, want), (shift, int((codes != want).sum()))
        rp.check(scale, ws, rp.E * ws + 2.0 ** -149, "scale")


def test_quant_rows_without_a_scale():
    X = torch.randn(6, 300, device="cuda")
    X[1] = 0.0
    X[2, 299] = math.nan
    X[3, 0] = -math.inf
    X[4] = -0.0
    for dtype in (BF16, FP32):
        x = X.to(dtype)
        codes, scale = torch.full((6, 300), 3, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
        rows.RowQuant(6, 300, dtype=dtype).run(rows.make_quant_args(X=x, codes=codes, scale=scale))
        assert bool((codes[1:5] == 0).all()) and bool(scale[2:4].isnan().all()) and bool((scale[[1, 4]] == 0).all())
        assert torch.equal(codes, rp.quant(x)[0])


# ---- product of codes ----

def i8_inputs(M, N, K, dtype, bias, residual, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    code = lambda *s: torch.randint(-128, 128, s, generator=gen, device="cuda").to(torch.int8)  # noqa: E731
    X, W = code(M, K), code(N, K)
    xs, ws = torch.rand(M, generator=gen, device="cuda") * 0.02 + 1e-3, torch.rand(N, generator=gen, device="cuda") * 0.02 / max(K, 1) ** 0.5
    return (X, W, xs, ws, normal(gen, (N,), dtype) if bias else None, normal(gen, (M, N), dtype) if residual else None)


def run_i8(X, W, xs, ws, b, R, act, dtype, tile=None, pads=(0, 0, 0, 0)):
    M, K, N = *X.shape, W.shape[0]
    lds = dict(ldx=K + pads[0], ldw=K + pads[1], ldy=N + pads[2], ldr=N + pads[3])
    lay = lambda t, ld, extra: padded(t, ld) if extra else t  # noqa: E731
    X, W = lay(X, lds["ldx"], pads[0]), lay(W, lds["ldw"], pads[1])
    Y, R = lay(torch.full((M, N), float("nan"), dtype=dtype, device="cuda"), lds["ldy"], pads[2]), lay(R, lds["ldr"], pads[3])
    plan = rows.Int8Linear(M, N, K, act=act, bias=b is not None, residual=R is not None, dtype=dtype, tile=tile, **lds)
    plan.run(rows.make_i8_args(X=X, W=W, x_scale=xs, w_scale=ws, bias=b, residual=R, Y=Y))
    if pads[2]:
        assert canary_ok(Y)
    return Y, plan


I8_SIZES = [(1, 8, 16), (1, 128, 128), (3, 136, 48), (16, 256, 4096), (17, 1000, 272), (64, 64, 64), (65, 72, 144), (129, 520, 1040),
            (256, 256, 256), (300, 776, 2064), (777, 264, 528), (1, 4096, 1040), (16, 1032, 11008), (1000, 2056, 144), (2, 24, 11008), (13, 264, 11008),
            (27, 520, 4112), (32, 1000, 4096), (19, 4200, 4096), (32, 16, 496), (33, 136, 2048), (5, 72, 131056)]


@pytest.mark.parametrize("tile", [None, rows.GE_I8_TILE_256, rows.GE_I8_TILE_128, rows.GE_I8_TILE_64])
@pytest.mark.parametrize("M,N,K", I8_SIZES)
def test_i8_sizes(M, N, K, tile):
    x = i8_inputs(M, N, K, FP32, False, False)
    Y, _ = run_i8(*x, "none", FP32, tile)
    rp.check(Y, *rp.int8(*x, "none", FP32), "Y")


@pytest.mark.parametrize("N", [8, 2040, 2048, 2056, 4096, 4104, 6144, 6152])
@pytest.mark.parametrize("M", [1, 4, 5, 17])
def test_i8_few_tokens_where_workgroups_change(M, N):
    x = i8_inputs(M, N, 528, BF16, True, True)
    Y, plan = run_i8(*x, "none", BF16, pads=(0, 0, 8, 16))
    assert ("few rows" in plan.describe()) == (M <= 5 or N <= 4096)
    rp.check(Y, *rp.int8(*x, "none", BF16), "Y")
    assert torch.equal(Y, run_i8(*x, "none", BF16, rows.GE_I8_TILE_64)[0])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,N,K", [(5, 520, 272), (150, 392, 528)])
def test_i8_epilogues(M, N, K, bias, residual, act, dtype):
    x = i8_inputs(M, N, K, dtype, bias, residual, seed=3)
    first = None
    for tile in (None, rows.GE_I8_TILE_256, rows.GE_I8_TILE_128, rows.GE_I8_TILE_64):
        Y, _ = run_i8(*x, act, dtype, tile, pads=(16, 32, 8, 16))
        rp.check(Y, *rp.int8(*x, act, dtype), "Y")
        if first is None:
            first = Y
        assert torch.equal(first, Y)               # the sums are exact: every tile gives the same bits


@pytest.mark.parametrize("M", [1, 20, 300])
def test_i8_largest_sums(M):
    """All codes -128 at the longest contraction: the sum is 2^31 - 2^18."""
    N, K = 264, (1 << 17) - 16
    X = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    W = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    W[1::2] = 127
    one = torch.ones(max(M, N), device="cuda")
    Y, _ = run_i8(X, W, one[:M], one[:N], None, None, "none", FP32)
    assert bool((Y[:, ::2].double() == float(128 * 128 * K)).all()) and bool((Y[:, 1::2].double() == float(torch.tensor(-128. * 127 * K).float())).all())


def test_i8_empty_and_not_finite():
    one = torch.ones(16, device="cuda")
    code = lambda *s: torch.ones(s, dtype=torch.int8, device="cuda")  # noqa: E731
    run_i8(code(0, 16), code(8, 16), one[:0], one[:8], None, None, "none", BF16)
    run_i8(code(4, 16), code(0, 16), one[:4], one[:0], None, None, "none", BF16)
    b = torch.arange(8, device="cuda").to(BF16)
    Y, _ = run_i8(code(4, 0), code(8, 0), one[:4], one[:8], b, None, "none", BF16)      # no contraction: the bias
    assert torch.equal(Y, b.expand(4, 8))
    for act in ("none", "relu", "gelu_tanh", "silu"):
        xs = one[:4].clone()
        xs[2] = math.nan
        Y, _ = run_i8(code(4, 16), code(8, 16), xs, one[:8], None, None, act, FP32)
        assert bool(Y[2].isnan().all()) and bool(Y[[0, 1, 3]].isfinite().all())


def test_i8_residual_in_place():
    M, N, K = 40, 264, 512
    x = i8_inputs(M, N, K, BF16, True, True, seed=8)
    Y, _ = run_i8(*x, "silu", BF16)
    R = x[5].clone()
    plan = rows.Int8Linear(M, N, K, act="silu", bias=True, residual=True)
    plan.run(rows.make_i8_args(X=x[0], W=x[1], x_scale=x[2], w_scale=x[3], bias=x[4], residual=R, Y=R))
    assert torch.equal(R, Y)

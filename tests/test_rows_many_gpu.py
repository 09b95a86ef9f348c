"""Row operators in calls whose outputs pass what the caches keep (other loads and stores are compiled for these) and
in calls of more rows than a grid has workgroups: every row shape and both types, against the 64-bit definitions or,
bit for bit, against the same rows in other calls."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import rows_parity as rp

pytestmark = pytest.mark.gpu

rows = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.rows")

BF16, FP32 = torch.bfloat16, torch.float32
LARGE = 64 << 20                                       # bytes of outputs
SEED, OFFSET, SITE = 21, (3 << 32) + 4, 2
WIDTHS = [264, 1024, 2048, 4096, 8192, 11008, 32768]   # one of every row shape


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def rng():
    return torch.tensor([SEED, OFFSET], dtype=torch.int64, device="cuda")


def rows_past_the_limit(d, size):
    return LARGE // (d * size) + 5


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def sample(M):
    """The first rows, the last ones and some between."""
    return sorted({*range(4), *range(M - 4, M), *range(5, M, max(1, M // 23))})


def factors(which, d, p):
    """What dropout multiplies the values of these rows with (d a multiple of eight)."""
    t, nb = round(p * rp.STEPS), d // 8
    at = (np.asarray(which, np.uint64)[:, None] * np.uint64(nb) + np.arange(nb, dtype=np.uint64)).astype(np.uint32).ravel()
    full = lambda v: np.full(at.shape, v & 0xFFFFFFFF, np.uint32)  # noqa: E731
    w = rp.philox((at, full(SITE), full(OFFSET), full(OFFSET >> 32)), (SEED, 0))
    half = np.stack([h for x in w for h in (x & np.uint32(0xFFFF), x >> np.uint32(16))], -1).reshape(len(which), d)
    return torch.from_numpy((half >= t) * (rp.STEPS / (rp.STEPS - t))).cuda()


def test_factors_of_some_rows_are_those_of_all():
    which = [0, 3, 16]
    assert torch.equal(factors(which, 40, 0.25).cpu(), rp.drop_factors(17, 40, 0.25, SEED, OFFSET, SITE)[which])


@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", WIDTHS)
def test_norm_of_many_rows(d, dtype, p):
    size = torch.finfo(dtype).bits // 8
    M = rows_past_the_limit(d, size)
    gen = torch.Generator("cuda").manual_seed(d)
    X, R, dY, dS = (normal(gen, (M, d), dtype, s) for s in (1.0, 2.0, 0.05, 0.05))
    gain, bias = normal(gen, (d,), dtype), normal(gen, (d,), dtype)
    e = lambda: torch.full((M, d), float("nan"), dtype=dtype, device="cuda")  # noqa: E731
    S, Y, Y1, dX, dR, dX1 = (e() for _ in range(6))
    mean, rstd, dgain, dbias, dgain1 = (torch.empty(k, device="cuda") for k in (M, M, d, d, d))
    plan = rows.LayerNorm(M, d, dtype=dtype, residual=True, dropout=p, site=SITE)
    common = dict(gain=gain, rng=rng())
    plan.forward(rows.make_norm_args(X=X, residual=R, S=S, Y=Y, bias=bias, mean=mean, rstd=rstd, **common))
    plan.forward(rows.make_norm_args(X=X, residual=R, Y=Y1, bias=bias, **common))
    assert torch.equal(Y, Y1)
    at = sample(M)
    f = factors(at, d, p) if p else None
    s, ts = rp.norm_sum(X[at], R[at], f)
    rp.check(S[at], s, ts, "S")
    ref, tol = rp.norm_forward(S, gain, bias, 1e-5)
    for n, got in (("Y", Y), ("mean", mean), ("rstd", rstd)):
        rp.check(got, ref[n], tol[n], (n, d))
    del ref, tol, Y1
    back = dict(S=S, mean=mean, rstd=rstd, dY=dY, dS=dS, **common)
    plan.backward(rows.make_norm_args(dX=dX, dR=dR, dgain=dgain, dbias=dbias, **back))
    plan.backward(rows.make_norm_args(dX=dX1, dgain=dgain1, **back))
    assert torch.equal(dX, dX1) and torch.equal(dgain, dgain1)
    ref, tol = rp.norm_backward(dY, S, dS, mean, rstd, gain, None)
    for n, got in (("dR", dR), ("dgain", dgain), ("dbias", dbias)):
        rp.check(got, ref[n], tol[n], (n, d))
    del ref, tol
    ref, tol = rp.norm_backward(dY[at], S[at], dS[at], mean[at], rstd[at], gain, f)
    rp.check(dX[at], ref["dX"], tol["dX"], "dX")


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [1024, 11008])
def test_dropout_of_many_rows(d, dtype, residual):
    M = rows_past_the_limit(d, torch.finfo(dtype).bits // 8)
    gen = torch.Generator("cuda").manual_seed(d)
    X, dY = normal(gen, (M, d), dtype), normal(gen, (M, d), dtype)
    R = normal(gen, (M, d), dtype) if residual else None
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    plan = rows.Dropout(M, d, 0.25, dtype=dtype, residual=residual, site=SITE)
    args = rows.make_dropout_args(X=X, residual=R, Y=Y, dY=dY, dX=dX, rng=rng())
    plan.forward(args)
    plan.backward(args)
    at = sample(M)
    f, half = factors(at, d, 0.25), rp.half_step(dtype)
    kept = X[at].double() * f
    want = kept + (R[at].double() if residual else 0)
    rp.check(Y[at], want, half * want.abs() + 3 * rp.E * (kept.abs() + want.abs()) + rp.TINY, "Y")
    want = dY[at].double() * f
    rp.check(dX[at], want, (half + 3 * rp.E) * want.abs() + rp.TINY, "dX")
    # rows that are not dense are computed by another instance
    wide = lambda t: torch.cat([t, t[:, :8]], 1)[:, :d]  # noqa: E731
    Y1, dX1 = wide(torch.empty_like(X)), wide(torch.empty_like(X))
    other = rows.Dropout(M, d, 0.25, dtype=dtype, residual=residual, site=SITE, ldy=d + 8, lddx=d + 8)
    other.forward(rows.make_dropout_args(X=X, residual=R, Y=Y1, rng=rng()))
    other.backward(rows.make_dropout_args(dY=dY, dX=dX1, rng=rng()))
    assert torch.equal(Y, Y1) and torch.equal(dX, dX1)


@pytest.mark.parametrize("gap", [0, 3, 8])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", WIDTHS)
def test_codes_of_many_rows(d, dtype, gap):
    """Codes of rows that lie dense, at odd addresses and at a pitch of their own."""
    M = rows_past_the_limit(d, 1)
    X = normal(torch.Generator("cuda").manual_seed(d), (M, d), dtype, 3.0)
    buf, scale = torch.full((M, d + gap), 77, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    codes = buf[:, :d]
    rows.RowQuant(M, d, dtype=dtype, ldq=d + gap).run(rows.make_quant_args(X=X, codes=codes, scale=scale))
    want, ws = rp.quant(X)
    assert torch.equal(codes, want) and bool((buf[:, d:] == 77).all())
    rp.check(scale, ws, rp.E * ws + 2.0 ** -149, "scale")


@pytest.mark.parametrize("M,d", [((4 << 20) + 5, 8), ((4 << 20) + 5, 9), ((1 << 20) + 3, 1029), ((1 << 20) + 3, 1032)])
def test_norm_of_more_rows_than_a_grid_has_workgroups(M, d):
    """A workgroup takes a second row (or four): the same bits as in calls of half the rows."""
    gen = torch.Generator("cuda").manual_seed(d)
    X = normal(gen, (M, d), BF16)
    gain, bias = normal(gen, (d,), BF16), normal(gen, (d,), BF16)
    Y, mean, rstd = torch.full_like(X, float("nan")), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    rows.LayerNorm(M, d).forward(rows.make_norm_args(X=X, Y=Y, gain=gain, bias=bias, mean=mean, rstd=rstd))
    for part in (slice(0, M // 2), slice(M // 2, M)):
        x = X[part]
        y, m, r = torch.empty_like(x), torch.empty(len(x), device="cuda"), torch.empty(len(x), device="cuda")
        rows.LayerNorm(len(x), d).forward(rows.make_norm_args(X=x, Y=y, gain=gain, bias=bias, mean=m, rstd=r))
        assert torch.equal(Y[part], y) and torch.equal(mean[part], m) and torch.equal(rstd[part], r)
    ref, tol = rp.norm_forward(X[-9:], gain, bias, 1e-5)
    rp.check(Y[-9:], ref["Y"], tol["Y"], "Y")

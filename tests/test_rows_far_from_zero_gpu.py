"""Layer norm's gradient of rows far from zero whose deviation is small: mean * rstd passes the largest fp32 number,
so what stands for places past the end of a row must not reach the row's sums."""
from __future__ import annotations

import pytest
import torch

from tests import rows_parity as rp

pytestmark = pytest.mark.gpu

rows = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.rows")

BF16, FP32 = torch.bfloat16, torch.float32
EPS, FAR = 1e-12, 2.0 ** 110                           # rstd of equal values 1e6: mean * rstd 1.3e39
# every row shape, filled and not, ragged and not
WIDTHS = [1, 3, 8, 9, 24, 512, 515, 520, 1021, 1024, 1032, 2048, 2056, 4095, 4096, 4104, 8192, 8200, 11007, 16384, 16392, 32761, 32768]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", WIDTHS)
def test_gradient_of_equal_values_far_from_zero(d, dtype):
    """Odd rows are FAR everywhere (their sums are exact: a power of two times a whole number below 2^24), even rows
    ordinary ones."""
    M, p, site = 9, 0.25, 6
    gen = torch.Generator("cuda").manual_seed(d)
    n = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(dtype)  # noqa: E731
    X, R, dY, dS = n(M, d), n(M, d), n(M, d), n(M, d)
    gain, bias = n(d), n(d)
    X[1::2], R[1::2] = 0.0, FAR
    rng = torch.tensor([11, 12], dtype=torch.int64, device="cuda")
    plan = rows.LayerNorm(M, d, eps=EPS, dtype=dtype, residual=True, dropout=p, site=site)
    e = lambda: torch.empty_like(X)  # noqa: E731
    S, Y, dX, dR = e(), e(), e(), e()
    mean, rstd, dgain, dbias = (torch.empty(k, device="cuda") for k in (M, M, d, d))
    plan.forward(rows.make_norm_args(X=X, residual=R, S=S, Y=Y, gain=gain, bias=bias, mean=mean, rstd=rstd, rng=rng))
    assert bool((mean[1::2] == FAR).all()) and torch.equal(Y[1::2], bias.expand_as(Y[1::2]))
    plan.backward(rows.make_norm_args(S=S, mean=mean, rstd=rstd, gain=gain, rng=rng, dY=dY, dS=dS, dX=dX, dR=dR, dgain=dgain,
                                      dbias=dbias))
    ref, tol = rp.norm_backward(dY, S, dS, mean, rstd, gain, rp.drop_factors(M, d, p, 11, 12, site).cuda())
    for name, got in (("dX", dX), ("dR", dR), ("dgain", dgain), ("dbias", dbias)):
        assert bool(got.isfinite().all()), (name, d)
        rp.check(got, ref[name], tol[name], (name, d))

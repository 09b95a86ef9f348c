"""The row operators where offsets pass 32 bits: the far end of the tensors is computed like the same
rows by themselves."""
from __future__ import annotations

import pytest
import torch

from tests import rows_parity as rp

pytestmark = pytest.mark.gpu

rows = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.rows")

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB of device memory")
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def far(M, d, ld, seed, n=40):
    """M rows ld apart (past 4 GB), zero but for the first and the last n."""
    buf = torch.zeros(M, ld, dtype=BF16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(seed)
    for part in (buf[:n, :d], buf[-n:, :d]):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    return buf[:, :d]


def test_norm_and_codes_past_4_gb():
    M, d, ld, n = 70001, 520, 40000, 40                # 5.6 GB of rows
    X = far(M, d, ld, 1)
    gen = torch.Generator("cuda").manual_seed(2)
    gain, bias = (torch.randn(d, generator=gen, device="cuda").to(BF16) for _ in range(2))
    S = torch.empty(M, ld, dtype=BF16, device="cuda")[:, :d]
    Y, mean, rstd = torch.empty(M, d, dtype=BF16, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    plan = rows.LayerNorm(M, d, dropout=0.5, ldx=ld, lds=ld, site=1)
    plan.forward(rows.make_norm_args(X=X, S=S, Y=Y, gain=gain, bias=bias, mean=mean, rstd=rstd, rng=rng))
    f = rp.drop_factors(M, d, 0.5, 3, 4, 1)[-n:].cuda()
    s, ts = rp.norm_sum(X[-n:], None, f)
    rp.check(S[-n:], s, ts, "S")
    ref, tol = rp.norm_forward(S[-n:], gain, bias, 1e-5)
    rp.check(Y[-n:], ref["Y"], tol["Y"], "Y")
    # gradients: only the far rows have any
    dY = torch.zeros(M, d, dtype=BF16, device="cuda")
    dY[-n:] = torch.randn(n, d, generator=gen, device="cuda").to(BF16)
    dX, dgain, dbias = torch.full((M, d), 7, dtype=BF16, device="cuda"), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    plan.backward(rows.make_norm_args(S=S, mean=mean, rstd=rstd, gain=gain, rng=rng, dY=dY, dX=dX, dgain=dgain, dbias=dbias))
    ref, tol = rp.norm_backward(dY[-n:], S[-n:], None, mean[-n:], rstd[-n:], gain, f)
    for k, got in (("dX", dX[-n:]), ("dgain", dgain), ("dbias", dbias)):
        rp.check(got, ref[k], tol[k], k)
    assert bool((dX[:-n] == 0).all())
    codes, scale = torch.full((M, d), 5, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    rows.RowQuant(M, d, ldx=ld).run(rows.make_quant_args(X=X, codes=codes, scale=scale))
    assert torch.equal(codes[-n:], rp.quant(X[-n:])[0]) and torch.equal(codes[:n], rp.quant(X[:n])[0])
    assert bool((codes[n:-n] == 0).all()) and bool((scale[n:-n] == 0).all())


@pytest.mark.parametrize("d,ld", [(70000, 70000), (70000, 70008), (69999, 69999)])
def test_dropout_past_2_32_values(d, ld):
    M, n = 61500, 2                                    # 4.3e9 values, dense and not
    X = torch.ones(M, ld, dtype=BF16, device="cuda")[:, :d]
    Y = torch.zeros(M, ld, dtype=BF16, device="cuda")[:, :d]
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    rows.Dropout(M, d, 0.5, ldx=ld, ldy=ld).forward(rows.make_dropout_args(X=X, Y=Y, rng=rng))
    # the last rows' blocks have counters of their own: drawn here from their place in the whole
    nb = -(-d // 8)
    import numpy as np
    at = np.arange((M - n) * nb, M * nb, dtype=np.uint64).astype(np.uint32)
    zero = np.zeros_like(at)
    w = rp.philox((at, zero, zero + np.uint32(4), zero), (3, 0))
    half = np.stack([h for x in w for h in (x & np.uint32(0xFFFF), x >> np.uint32(16))], -1).reshape(n, nb * 8)[:, :d]
    assert torch.equal(Y[-n:].float().cpu(), torch.from_numpy((half >= 32768) * np.float32(2)))
    share = float((Y[30000:30100] == 0).float().mean())
    assert abs(share - 0.5) < 0.002


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_int8_product_past_4_gb(dtype):
    """270,336 tokens of 8,192 outputs and, with a wide pitch, 4.3 GB of codes."""
    M, N, K, n = 270336, 8192 if dtype == BF16 else 4096, 64, 64
    gen = torch.Generator("cuda").manual_seed(3)
    X = torch.randint(-127, 128, (M, 16384), generator=gen, device="cuda", dtype=torch.int8)[:, :K]
    W = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(M, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
    Y = torch.zeros(M, N, dtype=dtype, device="cuda")
    plan = rows.Int8Linear(M, N, K, dtype=dtype, ldx=16384)
    plan.run(rows.make_i8_args(X=X, W=W, x_scale=xs, w_scale=ws, Y=Y))
    for part in (slice(0, n), slice(135000, 135000 + n), slice(M - n, M)):
        rp.check(Y[part], *rp.int8(X[part], W, xs[part], ws, None, None, "none", dtype), "Y")


def test_int8_weights_past_4_gb():
    """1,100,000 weight rows of 4,096 codes (4.5 GB), one token and a tile's worth of tokens."""
    N, K = 1_100_000, 4096
    gen = torch.Generator("cuda").manual_seed(4)
    W = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=gen, device="cuda")
    for M in (1, 40):
        X, xs = torch.randint(-127, 128, (M, K), generator=gen, device="cuda", dtype=torch.int8), torch.rand(M, device="cuda")
        Y = torch.zeros(M, N, dtype=BF16, device="cuda")
        rows.Int8Linear(M, N, K).run(rows.make_i8_args(X=X, W=W, x_scale=xs, w_scale=ws, Y=Y))
        for part in (slice(0, 200), slice(524288 - 100, 524288 + 100), slice(N - 200, N)):
            rp.check(Y[:, part], *rp.int8(X, W[part], xs, ws[part], None, None, "none", BF16), "Y")

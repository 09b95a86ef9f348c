"""The row operators in calls that their documentation allows and that are easy to get wrong: outputs over
inputs where rows are ragged, one tensor in two places, pointers at odd addresses, anything at all between rows, rows
with NaN next to others, contractions of no codes, one handle in two threads."""
from __future__ import annotations

import threading

import pytest
import torch

from tests import rows_parity as rp

pytestmark = pytest.mark.gpu

rows = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.rows")

BF16, FP32 = torch.bfloat16, torch.float32
TILES = [None, rows.GE_I8_TILE_256, rows.GE_I8_TILE_128, rows.GE_I8_TILE_64]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def odd(t):
    """The same values one element past an aligned address."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    return buf[1:].view(t.shape).copy_(t)


def between(t, ld, what):
    """The same rows ld apart, with `what` between them."""
    buf = torch.full((t.shape[0], ld), what, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def rng():
    return torch.tensor([11, 12], dtype=torch.int64, device="cuda")


def norm_inputs(M, d, dtype, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed + d)
    return [normal(gen, (M, d), dtype) for _ in range(4)] + [normal(gen, (d,), dtype) for _ in range(2)]


def norm_step(M, d, dtype, X, R, dY, dS, gain, bias, over=False, **ld):
    """Forward and backward; `over`: every output that may be an input is one."""
    plan = rows.LayerNorm(M, d, dtype=dtype, residual=True, dropout=0.25, site=4, **ld)
    mean, rstd, dgain, dbias = (torch.empty(n, device="cuda") for n in (M, M, d, d))
    e = lambda: torch.empty(M, d, dtype=dtype, device="cuda")  # noqa: E731
    S, Y, dX, dR = (R, X, dY, dS) if over else (e(), e(), e(), e())
    plan.forward(rows.make_norm_args(X=X, residual=R, S=S, Y=Y, gain=gain, bias=bias, mean=mean, rstd=rstd, rng=rng()))
    plan.backward(rows.make_norm_args(S=S, mean=mean, rstd=rstd, gain=gain, rng=rng(), dY=dY, dS=dS, dX=dX, dR=dR, dgain=dgain,
                                      dbias=dbias))
    return [S, Y, mean, rstd, dX, dR, dgain, dbias]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M,d", [(700, 9), (300, 515), (300, 1021), (300, 4095), (300, 8191), (270, 11007), (260, 32761)])
def test_norm_of_ragged_rows_over_its_inputs(M, d, dtype):
    X, R, dY, dS, gain, bias = norm_inputs(M, d, dtype)
    apart = norm_step(M, d, dtype, X.clone(), R.clone(), dY.clone(), dS.clone(), gain, bias)
    over = norm_step(M, d, dtype, X, R, dY, dS, gain, bias, over=True)
    assert all(torch.equal(a, b) for a, b in zip(apart, over))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M,d", [(40, 1000), (40, 1021), (5, 4104)])
def test_norm_at_odd_addresses(M, d, dtype):
    x = norm_inputs(M, d, dtype)
    plain = norm_step(M, d, dtype, *x)
    moved = norm_step(M, d, dtype, *[odd(t) for t in x])
    assert all(torch.equal(a, b) for a, b in zip(plain, moved))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [520, 1021])
def test_one_tensor_in_two_places(d, dtype):
    M = 50
    X, _, dY, _, gain, _ = norm_inputs(M, d, dtype)
    twice = norm_step(M, d, dtype, X, X, dY, dY, gain, gain)
    once = norm_step(M, d, dtype, X, X.clone(), dY, dY.clone(), gain, gain.clone())
    assert all(torch.equal(a, b) for a, b in zip(twice, once))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("d", [24, 1000, 1021, 4099, 16400])
def test_a_row_of_nan_stays_alone_and_nothing_between_rows_counts(d, dtype):
    """NaN in one row and in the gaps: every other row's outputs are those without them."""
    M, bad, ld = 70, 33, d + 5
    x = norm_inputs(M, d, dtype)
    clean = norm_step(M, d, dtype, *x)
    nan = float("nan")
    x = [between(t, ld, nan) if t.dim() == 2 else t for t in x]
    for t in x[:4]:
        t[bad] = nan
    names = dict.fromkeys(("ldx", "ldr", "lddy", "ldds"), ld)
    got = norm_step(M, d, dtype, *x, **names)
    others = torch.arange(M, device="cuda") != bad
    for a, b in list(zip(clean, got))[:6]:
        assert torch.equal(a[others], b[others])
    assert bool(got[1][bad].isnan().all()) and bool(got[6].isnan().all()) and bool(got[7].isnan().all())
    codes, scale = torch.empty(M, d, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    rows.RowQuant(M, d, dtype=dtype, ldx=ld).run(rows.make_quant_args(X=x[0], codes=codes, scale=scale))
    want = rp.quant(norm_inputs(M, d, dtype)[0])
    assert torch.equal(codes[others], want[0][others]) and bool((codes[bad] == 0).all())
    assert bool(scale[bad].isnan()) and bool(scale[others].isfinite().all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M,d", [(3000, 9), (700, 1021), (700, 1024), (40, 11007)])
def test_dropout_over_its_inputs(M, d, dtype):
    gen = torch.Generator("cuda").manual_seed(d)
    X, R = normal(gen, (M, d), dtype), normal(gen, (M, d), dtype)
    plan = rows.Dropout(M, d, 0.3, dtype=dtype, residual=True)
    Y = torch.empty_like(X)
    plan.forward(rows.make_dropout_args(X=X, residual=R, Y=Y, rng=rng()))
    for over in (0, 1):
        t = [X.clone(), R.clone()]
        plan.forward(rows.make_dropout_args(X=t[0], residual=t[1], Y=t[over], rng=rng()))
        assert torch.equal(t[over], Y)
    dX, dY = torch.empty_like(X), X.clone()
    plan.backward(rows.make_dropout_args(dY=X, dX=dX, rng=rng()))
    plan.backward(rows.make_dropout_args(dY=dY, dX=dY, rng=rng()))
    assert torch.equal(dX, dY)


def i8_inputs(M, N, K, dtype, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed + M)
    code = lambda *s: torch.randint(-127, 128, s, generator=gen, device="cuda", dtype=torch.int8)  # noqa: E731
    return (code(M, K), code(N, K), torch.rand(M, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda"),
            normal(gen, (N,), dtype), normal(gen, (M, N), dtype, 100.0))


def i8(x, dtype, act="none", tile=None, Y=None, **ld):
    X, W, xs, ws, b, R = x
    M, K, N = *X.shape, W.shape[0]
    if Y is None:
        Y = torch.empty(M, N, dtype=dtype, device="cuda")
    plan = rows.Int8Linear(M, N, K, act=act, bias=True, residual=True, dtype=dtype, tile=tile, **ld)
    plan.run(rows.make_i8_args(X=X, W=W, x_scale=xs, w_scale=ws, bias=b, residual=R, Y=Y))
    return Y


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("M,N,K", [(1, 264, 512), (5, 520, 1040), (20, 4104, 528), (32, 1032, 272), (27, 520, 8192), (300, 776, 1040), (600, 520, 528)])
def test_i8_over_its_residual_and_scales_at_odd_addresses(M, N, K, dtype):
    x = i8_inputs(M, N, K, dtype)
    Y = i8(x, dtype, "silu")
    R = x[5].clone()
    got = i8((x[0], x[1], odd(x[2]), odd(x[3]), x[4], R), dtype, "silu", Y=R)
    assert torch.equal(got, Y)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M", [3, 30, 300])
def test_i8_nothing_between_rows_counts(M, tile, dtype):
    N, K = 264, 528
    x = i8_inputs(M, N, K, dtype)
    Y = i8(x, dtype, "gelu_tanh", tile)
    moved = (between(x[0], 560, 99), between(x[1], 576, 99), x[2], x[3], x[4], between(x[5], 280, float("nan")))
    assert torch.equal(Y, i8(moved, dtype, "gelu_tanh", tile, ldx=560, ldw=576, ldr=280))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M", [2, 40, 300])
def test_i8_of_no_codes(M, tile, dtype):
    """K = 0: act(bias) + R."""
    x = i8_inputs(M, 264, 0, dtype)
    rp.check(i8(x, dtype, "relu", tile), *rp.int8(*x, "relu", dtype), "Y")


def test_one_handle_in_two_threads():
    """Calls only read the handle: two threads, each with its own stream, tensors and workspace."""
    M, d = 4000, 1000
    x = norm_inputs(M, d, BF16)
    plan = rows.LayerNorm(M, d)
    X, dY, gain = x[0], x[2], x[4]
    size = plan._workspace_size()
    results, errors = {}, []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                out = [torch.empty(M, d, dtype=BF16, device="cuda") for _ in range(2)]
                vec = [torch.empty(n, device="cuda") for n in (M, M, d, d)]
                args = rows.make_norm_args(X=X, S=X, gain=gain, Y=out[0], mean=vec[0], rstd=vec[1], dY=dY, dX=out[1], dgain=vec[2],
                                           dbias=vec[3], workspace=torch.zeros(size, dtype=torch.uint8, device="cuda"))
                forward = rows.make_norm_args(X=X, gain=gain, Y=out[0], mean=vec[0], rstd=vec[1])
                for _ in range(50):
                    plan.forward(forward)
                    plan.backward(args)
                torch.cuda.current_stream().synchronize()
                results[k] = out + vec
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    work("alone")
    want = results["alone"]
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(results[k], want))

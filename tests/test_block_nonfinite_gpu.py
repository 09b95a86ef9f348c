"""NaN gates in the feed-forward block reach what depends on them, and nothing else, with every
activation and every kernel."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

block = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.block")

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(BF16)


def weights(gen, d, h, layout):
    wi, wo = ((d, h), (h, d)) if layout == "kn" else ((h, d), (d, h))
    return normal(gen, *wi, std=d ** -0.5), normal(gen, *wi, std=d ** -0.5), normal(gen, *wo, std=h ** -0.5)


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,d,h,tile", [(20, 64, 136, None), (20, 64, 136, 0), (20, 64, 136, 1), (20, 64, 136, 2),
                                        (3, 2048, 4104, None)])
def test_nan_gates_forward(M, d, h, tile, layout, act):
    gen = torch.Generator("cuda").manual_seed(M + d)
    X, (Wg, Wu, Wd) = normal(gen, M, d), weights(gen, d, h, layout)
    plan = block.GatedFFN(M, d, h, act=act, w_layout=layout, tile=tile)

    def run():
        Y = torch.empty(M, d, device="cuda", dtype=BF16)
        plan.forward(block.make_ffn_args(X=X, Wg=Wg, Wu=Wu, Wd=Wd, Y=Y))
        return Y
    clean = run()
    assert clean.isfinite().all()
    # one gate column: every row has a NaN gate
    j = h - 3
    (Wg[:, j] if layout == "kn" else Wg[j]).fill_(math.nan)
    assert run().isnan().all()
    # one row of X
    (Wg[:, j] if layout == "kn" else Wg[j]).fill_(0)
    clean = run()
    X[1, 5] = math.nan
    got = run()
    assert got[1].isnan().all()
    rest = [r for r in range(M) if r != 1]
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("tile", [None, 0, 1, 2])
def test_nan_gates_backward(tile, layout, act):
    M, d, h, r, j = 20, 64, 136, 7, 131
    gen = torch.Generator("cuda").manual_seed(5)
    X, (Wg, Wu, Wd) = normal(gen, M, d), weights(gen, d, h, layout)
    G, U, dY = normal(gen, M, h), normal(gen, M, h), normal(gen, M, d)
    plan = block.GatedFFN(M, d, h, act=act, w_layout=layout, save=True, tile=tile)

    def run():
        out = dict(dX=torch.empty_like(X), dWg=torch.empty_like(Wg), dWu=torch.empty_like(Wu), dWd=torch.empty_like(Wd))
        plan.backward(block.make_ffn_args(X=X, Wg=Wg, Wu=Wu, Wd=Wd, G=G, U=U, dY=dY, **out))
        if layout == "nk":
            out = {k: v if k == "dX" else v.t() for k, v in out.items()}
        return out
    clean = run()
    G[r, j] = math.nan
    got = run()
    assert got["dX"][r].isnan().all() and got["dWu"][:, j].isnan().all() and got["dWd"][j].isnan().all()
    # the slope at NaN is NaN; ReLU's is 0 wherever the gate is not above zero, and no activation's is 1
    if act in ("gelu_tanh", "silu"):
        assert got["dWg"][:, j].isnan().all()
    else:
        assert got["dWg"].isfinite().all()
    rows, cols = [i for i in range(M) if i != r], [i for i in range(h) if i != j]
    assert torch.equal(got["dX"][rows], clean["dX"][rows])
    for k in ("dWg", "dWu"):
        assert torch.equal(got[k][:, cols], clean[k][:, cols]), k
    assert torch.equal(got["dWd"][cols], clean["dWd"][cols])

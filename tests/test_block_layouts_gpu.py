"""Layouts of the rotation's inputs that the other tests leave out, on the GPU: repeated elements."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

block = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.block")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 20])
@pytest.mark.parametrize("kind", ["heads", "tokens", "both"])
def test_expanded_inputs(kind, D, dtype):
    """One head for all heads, one token for all tokens: as if every element had a place of its own."""
    T, H = 300, 4
    gen = torch.Generator("cuda").manual_seed(6)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    q = r(1 if kind != "heads" else T, 1 if kind != "tokens" else H, D).expand(T, H, D)
    k = r(T, 2, D)
    common = dict(k=k, gain_q=r(D), gain_k=r(D), positions=torch.arange(T, device="cuda"),
                  inv_freq=block.rotary_frequencies(D)[0].cuda())
    dout = dict(dq_out=r(T, H, D), dk_out=r(T, 2, D))
    results = []
    for x in (q, q.contiguous()):
        plan = block.QKRotary(T, H, 2, D, q_strides=x.stride()[:2], dtype=dtype)
        e = lambda *s: torch.empty(s, device="cuda", dtype=dtype)  # noqa: E731
        out = dict(q_out=e(T, H, D), k_out=e(T, 2, D))
        grads = dict(dq=e(T, H, D), dk=e(T, 2, D), dgain_q=torch.empty(D, device="cuda"), dgain_k=torch.empty(D, device="cuda"))
        plan.forward(block.make_qk_args(q=x, **common, **out))
        plan.backward(block.make_qk_args(q=x, **common, **dout, **grads))
        results.append([*out.values(), *grads.values()])
    for a, b in zip(*results):
        assert torch.equal(a, b)

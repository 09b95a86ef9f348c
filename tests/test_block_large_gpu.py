"""The block operators where byte offsets pass 32 bits: the far end of the tensors is computed like the
same rows by themselves."""
from __future__ import annotations

import math

import pytest
import torch

from tests import block_parity as bp

pytestmark = pytest.mark.gpu

block = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.block")

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


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_feed_forward_past_4_gb(layout):
    """270,336 rows of 8,192 hidden values (4.4 GB each of G, U, H, dG and dU).  Only the last 64 rows have an
    output gradient, so the weight gradients are those of these rows alone, bit for bit: the other
    rows add zeros, and 64 rows are whole slots of the contraction."""
    M, d, h, n = 270336, 64, 8192, 64
    gen = torch.Generator("cuda").manual_seed(1)
    r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(BF16)  # noqa: E731
    wi, wo = ((d, h), (h, d)) if layout == "kn" else ((h, d), (d, h))
    X, Wg, Wu, Wd = r(M, d), r(*wi, std=0.1), r(*wi, std=0.1), r(*wo, std=0.02)
    e = lambda *s: torch.empty(s, device="cuda", dtype=BF16)  # noqa: E731
    tile = block.GE_FFN_TILE_256
    G, U, Y, dX = e(M, h), e(M, h), e(M, d), e(M, d)
    dW = [e(*wi), e(*wi), e(*wo)]
    dY = torch.zeros(M, d, device="cuda", dtype=BF16)
    dY[-n:] = r(n, d, std=0.1)
    plan = block.GatedFFN(M, d, h, w_layout=layout, save=True, tile=tile)
    args = dict(Wg=Wg, Wu=Wu, Wd=Wd)
    a = block.make_ffn_args(X=X, Y=Y, G=G, U=U, dY=dY, dX=dX, dWg=dW[0], dWu=dW[1], dWd=dW[2], **args)
    plan.forward(a)
    plan.backward(a)
    small = block.GatedFFN(n, d, h, w_layout=layout, save=True, tile=tile)
    g, u, y, dx = e(n, h), e(n, h), e(n, d), e(n, d)
    dw = [e(*wi), e(*wi), e(*wo)]
    b = block.make_ffn_args(X=X[-n:], Y=y, G=g, U=u, dY=dY[-n:], dX=dx, dWg=dw[0], dWu=dw[1], dWd=dw[2], **args)
    small.forward(b)
    small.backward(b)
    for big, one in ((G, g), (U, u), (Y, y), (dX, dx)):
        assert torch.equal(big[-n:], one)
    for big, one in zip(dW, dw):
        assert torch.equal(big, one)
    assert (dX[:-n] == 0).all()
    ref, tol = bp.ffn_forward(X[-n:], Wg, Wu, Wd, "silu", layout)
    bp.check(Y[-n:], ref["Y"], tol["Y"], "Y")


def test_rotation_past_4_gb():
    T, stride, hq, hk, D = 70001, 40000, 4, 2, 128           # 5.6 GB of rows
    rows = torch.zeros(T, stride, device="cuda", dtype=BF16)
    q, k = rows[:, 1024:1024 + hq * D].view(T, hq, D), rows[:, -hk * D:].view(T, hk, D)
    gen = torch.Generator("cuda").manual_seed(2)
    q.copy_(torch.randn(q.shape, generator=gen, device="cuda"))
    k.copy_(torch.randn(k.shape, generator=gen, device="cuda"))
    gain = torch.ones(D, device="cuda", dtype=BF16)
    pos, (inv, amp) = torch.arange(T, device="cuda"), block.rotary_frequencies(D)
    inv = inv.cuda()
    want = {w: bp.qk(x[-50:], None, gain, pos[-50:], inv, amp, D, "half", 1e-6) for w, x in (("q", q), ("k", k))}
    st = dict(q_strides=q.stride()[:2], k_strides=k.stride()[:2], q_out_strides=q.stride()[:2], k_out_strides=k.stride()[:2])
    block.QKRotary(T, hq, hk, D, **st).forward(block.make_qk_args(q=q, k=k, q_out=q, k_out=k, positions=pos, inv_freq=inv,
                                                                  gain_q=gain, gain_k=gain))
    bp.check(q[-50:], *want["q"], "q")
    bp.check(k[-50:], *want["k"], "k")
    assert (rows[:, :1024] == 0).all() and (rows[:, 1024 + hq * D:-hk * D] == 0).all()


def test_clipping_past_2_32_values():
    n = 2 ** 32 + 12345
    g = torch.zeros(n, device="cuda", dtype=BF16)
    g[-1000:] = 0.5
    g[2 ** 31 - 3:2 ** 31 + 3] = 2.0
    want = math.sqrt(1000 * 0.25 + 6 * 4.0)
    norm = torch.empty(1, device="cuda")
    plan = block.GradClip([g[:5], g[5:]])
    plan.run(block.make_clip_args([g[:5], g[5:]], [g[:5], g[5:]], norm=norm, max_norm=1.0))
    assert abs(float(norm) - want) <= want * 1.001 * bp.E
    f = 1.0 / (want + 1e-6)
    for part, v in ((g[-1000:], 0.5 * f), (g[2 ** 31 - 3:2 ** 31 + 3], 2.0 * f)):
        assert ((part.double() - v).abs() <= v * (bp.U + 4 * bp.E)).all()
    assert float(g[:2 ** 31 - 3].abs().max()) == 0 and float(g[2 ** 31 + 3:-1000].abs().max()) == 0

"""The transformer-block operators run together, as one training step of a block uses them: the
RMS-scaled QKV product of the fused library, the query/key norm with rotation in place on its output,
the feed-forward block forward and backward, the rotation's gradient, and the clipping of all
gradients in place.  Each stage is checked against its 64-bit definition on the inputs it was given."""
from __future__ import annotations

import math

import pytest
import torch

from tests import block_parity as bp

pytestmark = pytest.mark.gpu

ge = pytest.importorskip("gemm_epilogue_transformer_tiled_amd")
block = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.block")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


class Step:
    """One block of width d with hq query and hk key heads of D values, hidden width h, on T tokens."""

    def __init__(self, T, d, hq, hk, D, h, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).bfloat16()  # noqa: E731
        self.T, self.d, self.hq, self.hk, self.D, self.h = T, d, hq, hk, D, h
        width = (hq + 2 * hk) * D
        self.x, self.wqkv = r(T, d), r(d, width, std=d ** -0.5)
        self.gq, self.gk = r(D), r(D)
        self.Wg, self.Wu, self.Wd = r(d, h, std=d ** -0.5), r(d, h, std=d ** -0.5), r(h, d, std=h ** -0.5)
        self.pos = torch.arange(T, device="cuda")
        self.inv, self.amplitude = block.rotary_frequencies(D, scaling="by_parts", factor=4.0)
        self.inv = self.inv.cuda()
        self.dY, self.dq_out, self.dk_out = r(T, d, std=0.05), r(T, hq, D, std=0.05), r(T, hk, D, std=0.05)
        e = lambda *s: torch.empty(s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.qkv, self.raw = e(T, width), e(T, width)
        self.Y, self.G, self.U, self.dX = e(T, d), e(T, h), e(T, h), e(T, d)
        self.dqkv = torch.zeros(T, width, device="cuda", dtype=torch.bfloat16)
        self.dWg, self.dWu, self.dWd = e(d, h), e(d, h), e(h, d)
        self.dgq, self.dgk = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
        self.grads = [self.dWg, self.dWu, self.dWd, self.dgq, self.dgk]
        self.norm = torch.empty(1, device="cuda")
        # plans and packs, made once
        self.product = ge.Plan(ge.make_desc(1, T, width, d, ge.make_ops([("row_rms", 1e-6)])))
        self.product_args = ge.make_args(A=self.x, B=self.wqkv, Y=self.qkv)
        q, k = self.heads(self.qkv)
        dq, dk = self.heads(self.dqkv)
        rq, rk = self.heads(self.raw)
        st = dict(q_strides=q.stride()[:2], k_strides=k.stride()[:2])
        common = dict(positions=self.pos, inv_freq=self.inv, amplitude=self.amplitude, gain_q=self.gq, gain_k=self.gk)
        self.rotary = block.QKRotary(T, hq, hk, D, q_out_strides=q.stride()[:2], k_out_strides=k.stride()[:2], **st)
        self.rotary_args = block.make_qk_args(q=q, k=k, q_out=q, k_out=k, **common)
        self.rotary_grad = block.QKRotary(T, hq, hk, D, **st)
        self.rotary_grad_args = block.make_qk_args(q=rq, k=rk, dq_out=self.dq_out, dk_out=self.dk_out, dq=dq, dk=dk,
                                                   dgain_q=self.dgq, dgain_k=self.dgk, **common)
        self.ffn = block.GatedFFN(T, d, h, residual=True, save=True)
        self.ffn_args = block.make_ffn_args(X=self.x, Wg=self.Wg, Wu=self.Wu, Wd=self.Wd, residual=self.x, Y=self.Y, G=self.G,
                                            U=self.U, dY=self.dY, dX=self.dX, dWg=self.dWg, dWu=self.dWu, dWd=self.dWd)
        self.clip = block.GradClip(self.grads)
        self.clip_args = block.make_clip_args(self.grads, self.grads, norm=self.norm, max_norm=1.0)

    def heads(self, packed):
        a, b = self.hq * self.D, (self.hq + self.hk) * self.D
        return packed[:, :a].view(self.T, self.hq, self.D), packed[:, a:b].view(self.T, self.hk, self.D)

    def forward(self):
        self.product.run(self.product_args)
        self.raw.copy_(self.qkv)                       # the rotation's gradient needs its inputs
        self.rotary.forward(self.rotary_args)
        self.ffn.forward(self.ffn_args)

    def backward(self):
        self.ffn.backward(self.ffn_args)
        self.rotary_grad.backward(self.rotary_grad_args)

    def run(self):
        self.forward()
        self.backward()
        self.clip.run(self.clip_args)


@pytest.mark.parametrize("T,d,hq,hk,D,h", [(1, 256, 4, 2, 64, 520), (77, 264, 3, 1, 88, 712), (600, 512, 8, 2, 64, 1416)])
def test_training_step(T, d, hq, hk, D, h):
    s = Step(T, d, hq, hk, D, h)
    s.forward()
    values = s.raw[:, (hq + hk) * D:].clone()
    for w, gain, out, raw in zip("qk", (s.gq, s.gk), s.heads(s.qkv), s.heads(s.raw)):
        bp.check(out, *bp.qk(raw, None, gain, s.pos, s.inv, s.amplitude, D, "half", 1e-6), w)
    assert torch.equal(s.qkv[:, (hq + hk) * D:], values)
    ref, tol = bp.ffn_forward(s.x, s.Wg, s.Wu, s.Wd, "silu", "kn", s.x)
    for k, v in (("Y", s.Y), ("G", s.G), ("U", s.U)):
        bp.check(v, ref[k], tol[k], k)
    s.backward()
    ref, tol = bp.ffn_backward(s.x, s.Wg, s.Wu, s.Wd, s.G, s.U, s.dY, "silu", "kn")
    for k in ref:
        bp.check(getattr(s, k), ref[k], tol[k], k)
    for w, gain, d_out, raw, dx, dg in zip("qk", (s.gq, s.gk), (s.dq_out, s.dk_out), s.heads(s.raw), s.heads(s.dqkv), (s.dgq, s.dgk)):
        want, t, wg, tg = bp.qk(raw, d_out, gain, s.pos, s.inv, s.amplitude, D, "half", 1e-6)
        bp.check(dx, want, t, "d" + w)
        bp.check(dg, wg, tg, "dgain_" + w)
    assert (s.dqkv[:, (hq + hk) * D:] == 0).all()
    before = [g.double() for g in s.grads]
    s.clip.run(s.clip_args)
    norm = math.sqrt(sum(float(g.square().sum()) for g in before))
    assert abs(float(s.norm) - norm) <= norm * 1.001 * bp.E
    f = min(1.0, 1.0 / (norm + 1e-6))
    for g, b in zip(s.grads, before):
        bp.check(g, b * f, (b * f).abs() * (bp.half_step(g.dtype) + 4 * bp.E) + bp.TINY, "clipped")


def test_training_step_captured():
    """The whole step in one graph, replayed on new inputs, with eager steps between the replays."""
    s, t = Step(200, 264, 4, 2, 64, 520, seed=1), Step(200, 264, 4, 2, 64, 520, seed=1)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    gen = torch.Generator("cuda").manual_seed(9)
    for _ in range(4):
        x = torch.randn(s.x.shape, generator=gen, device="cuda")
        s.x.copy_(x)
        t.x.copy_(x)
        t.run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((s.Y, s.dX, s.qkv, s.dqkv, s.norm, *s.grads), (t.Y, t.dX, t.qkv, t.dqkv, t.norm, *t.grads)):
            assert torch.equal(a, b)

"""The row operators run together with the products around them, as a model uses them: a training step through
dropout, residual and norm between two products, forward and backward, eager and captured; and a serving
chain of norm, codes and int8 products.  Each stage is checked against its 64-bit definition on the inputs it
was given, and the step's gradients against those of the whole."""
from __future__ import annotations

import pytest
import torch

from tests import block_parity as bp
from tests import rows_parity as rp

pytestmark = pytest.mark.gpu

ge = pytest.importorskip("gemm_epilogue_transformer_tiled_amd")
block = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.block")
rows = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.rows")

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


class Step:
    """x -> product -> dropout, residual, norm -> feed-forward block -> dropout and residual, and back; the
    gradients of the block's weights, the gain and the bias are clipped at the end."""

    P1, P2 = 0.1, 0.3

    def __init__(self, T, d, h, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(BF16)  # noqa: E731
        e = lambda *s, t=BF16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.T, self.d, self.h = T, d, h
        self.rng = torch.tensor([1234567890123, 1 << 40], dtype=torch.int64, device="cuda")
        self.x, self.res, self.W = r(T, d), r(T, d), r(d, d, std=d ** -0.5)
        self.gain, self.bias = r(d, std=0.2) + 1, r(d, std=0.2)
        self.Wg, self.Wu, self.Wd = r(d, h, std=d ** -0.5), r(d, h, std=d ** -0.5), r(h, d, std=h ** -0.5)
        self.dout = r(T, d, std=0.1)
        self.a, self.S, self.n, self.f, self.out = e(T, d), e(T, d), e(T, d), e(T, d), e(T, d)
        self.mean, self.rstd, self.G, self.U = e(T, t=FP32), e(T, t=FP32), e(T, h), e(T, h)
        self.df, self.dn, self.da, self.dres = e(T, d), e(T, d), e(T, d), e(T, d)
        self.dWg, self.dWu, self.dWd = e(d, h), e(d, h), e(h, d)
        self.dgain, self.dbias, self.norm_of = e(d, t=FP32), e(d, t=FP32), e(1, t=FP32)
        self.product = ge.Plan(ge.make_desc(1, T, d, d, ge.make_ops([])))
        self.product_args = ge.make_args(A=self.x, B=self.W, Y=self.a)
        self.norm = rows.LayerNorm(T, d, residual=True, dropout=self.P1, site=0)
        self.norm_args = rows.make_norm_args(X=self.a, residual=self.res, S=self.S, Y=self.n, gain=self.gain, bias=self.bias,
                                             mean=self.mean, rstd=self.rstd, rng=self.rng, dY=self.dn, dS=self.dout, dX=self.da,
                                             dR=self.dres, dgain=self.dgain, dbias=self.dbias)
        self.ffn = block.GatedFFN(T, d, h, save=True)
        self.ffn_args = block.make_ffn_args(X=self.n, Wg=self.Wg, Wu=self.Wu, Wd=self.Wd, Y=self.f, G=self.G, U=self.U, dY=self.df,
                                            dX=self.dn, dWg=self.dWg, dWu=self.dWu, dWd=self.dWd)
        self.drop = rows.Dropout(T, d, self.P2, residual=True, site=1)
        self.drop_args = rows.make_dropout_args(X=self.f, residual=self.S, Y=self.out, dY=self.dout, dX=self.df, rng=self.rng)
        self.grads = [self.dWg, self.dWu, self.dWd, self.dgain, self.dbias]
        self.clip = block.GradClip(self.grads)
        self.clip_args = block.make_clip_args(self.grads, self.grads, norm=self.norm_of, max_norm=1e6)

    def run(self):
        self.product.run(self.product_args)
        self.norm.forward(self.norm_args)
        self.ffn.forward(self.ffn_args)
        self.drop.forward(self.drop_args)
        self.drop.backward(self.drop_args)
        self.ffn.backward(self.ffn_args)
        self.norm.backward(self.norm_args)
        self.clip.run(self.clip_args)

    def results(self):
        return [self.a, self.S, self.n, self.f, self.out, self.df, self.dn, self.da, self.dres, *self.grads, self.norm_of]


def factors(s, p, site):
    seed, offset = (int(v) for v in s.rng)
    return rp.drop_factors(s.T, s.d, p, seed, offset, site).cuda()


@pytest.mark.parametrize("T,d,h", [(1, 264, 520), (77, 264, 712), (600, 1032, 1416)])
def test_training_step(T, d, h):
    s = Step(T, d, h)
    s.run()
    f1, f2 = factors(s, s.P1, 0), factors(s, s.P2, 1)
    rp.check(s.S, *rp.norm_sum(s.a, s.res, f1), "S")
    ref, tol = rp.norm_forward(s.S, s.gain, s.bias, 1e-5)
    rp.check(s.n, ref["Y"], tol["Y"], "n")
    ref, tol = bp.ffn_forward(s.n, s.Wg, s.Wu, s.Wd, "silu", "kn")
    bp.check(s.f, ref["Y"], tol["Y"], "f")
    rp.check(s.out, *rp.norm_sum(s.f, s.S, f2), "out")
    want = rp.drop(s.dout.double(), f2)
    rp.check(s.df, want, (rp.half_step(BF16) + 3 * rp.E) * want.abs() + rp.TINY, "df")
    ref, tol = bp.ffn_backward(s.n, s.Wg, s.Wu, s.Wd, s.G, s.U, s.df, "silu", "kn")
    for k, got in (("dX", s.dn), ("dWg", s.dWg), ("dWu", s.dWu), ("dWd", s.dWd)):
        bp.check(got, ref[k], tol[k], k)
    ref, tol = rp.norm_backward(s.dn, s.S, s.dout, s.mean, s.rstd, s.gain, f1)
    for k, got in (("dX", s.da), ("dR", s.dres), ("dgain", s.dgain), ("dbias", s.dbias)):
        rp.check(got, ref[k], tol[k], k)


def test_the_steps_gradients_are_those_of_the_whole():
    """Against autograd in 64 bits on the CPU, through all stages: some twenty roundings to bf16 lie on the way to each
    gradient, sqrt(20) 2^-8 = 1.7 % of its norm if they are independent; twice that is allowed."""
    s = Step(96, 136, 264, seed=3)
    s.run()
    f1, f2 = factors(s, s.P1, 0).cpu(), factors(s, s.P2, 1).cpu()
    w = {k: getattr(s, k).double().cpu().requires_grad_(True) for k in ("x", "res", "W", "gain", "bias", "Wg", "Wu", "Wd")}
    a = w["x"] @ w["W"]
    a.retain_grad()
    S = w["res"] + a * f1
    c = S - S.mean(1, keepdim=True)
    n = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * w["gain"] + w["bias"]
    g = n @ w["Wg"]
    out = S + ((g * torch.sigmoid(g) * (n @ w["Wu"])) @ w["Wd"]) * f2
    out.backward(s.dout.double().cpu())
    for got, want in ((s.out, out), (s.da, a.grad), (s.dres, w["res"].grad), (s.dgain, w["gain"].grad), (s.dbias, w["bias"].grad),
                      (s.dWg, w["Wg"].grad), (s.dWu, w["Wu"].grad), (s.dWd, w["Wd"].grad)):
        off = (got.double().cpu() - want).norm() / want.norm()
        assert off < 0.035, float(off)


def test_training_step_captured():
    """The whole step in one graph, with a new mask at every replay, and eager steps between the replays."""
    s, t = Step(200, 264, 520, seed=1), Step(200, 264, 520, seed=1)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.rng[1] += 1
        s.run()
    s.rng.copy_(t.rng)
    gen = torch.Generator("cuda").manual_seed(9)
    masks = []
    for _ in range(4):
        x = torch.randn(s.x.shape, generator=gen, device="cuda")
        s.x.copy_(x)
        t.x.copy_(x)
        t.rng[1] += 1
        t.run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(s.results(), t.results()):
            assert torch.equal(a, b)
        masks.append(s.df == 0)
    assert not torch.equal(masks[0], masks[1])


class Serve:
    """norm with residual -> codes per token -> int8 product with bias and GELU -> codes -> int8 product with
    residual, for T tokens; the weights are coded per channel once."""

    def __init__(self, T, d, h, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(BF16)  # noqa: E731
        e = lambda *s, t=BF16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.T, self.d, self.h = T, d, h
        self.x, self.res, self.gain, self.bias, self.b1 = r(T, d), r(T, d), r(d, std=0.2) + 1, r(d, std=0.2), r(h, std=0.2)
        self.w1, self.w2 = r(h, d, std=d ** -0.5), r(d, h, std=h ** -0.5)
        self.c1, self.s1, self.c2, self.s2 = e(h, d, t=torch.int8), e(h, t=FP32), e(d, h, t=torch.int8), e(d, t=FP32)
        for w, c, sc in ((self.w1, self.c1, self.s1), (self.w2, self.c2, self.s2)):
            rows.RowQuant(*w.shape).run(rows.make_quant_args(X=w, codes=c, scale=sc))
        self.S, self.n, self.u, self.y = e(T, d), e(T, d), e(T, h), e(T, d)
        self.cn, self.sn, self.cu, self.su = e(T, d, t=torch.int8), e(T, t=FP32), e(T, h, t=torch.int8), e(T, t=FP32)
        self.calls = [
            (rows.LayerNorm(T, d, residual=True), "forward", rows.make_norm_args(X=self.x, residual=self.res, S=self.S, Y=self.n,
                                                                                gain=self.gain, bias=self.bias)),
            (rows.RowQuant(T, d), "run", rows.make_quant_args(X=self.n, codes=self.cn, scale=self.sn)),
            (rows.Int8Linear(T, h, d, act="gelu_tanh", bias=True), "run",
             rows.make_i8_args(X=self.cn, W=self.c1, x_scale=self.sn, w_scale=self.s1, bias=self.b1, Y=self.u)),
            (rows.RowQuant(T, h), "run", rows.make_quant_args(X=self.u, codes=self.cu, scale=self.su)),
            (rows.Int8Linear(T, d, h, residual=True), "run",
             rows.make_i8_args(X=self.cu, W=self.c2, x_scale=self.su, w_scale=self.s2, residual=self.S, Y=self.y))]

    def run(self):
        for plan, call, args in self.calls:
            getattr(plan, call)(args)


@pytest.mark.parametrize("T,d,h", [(1, 1024, 4096), (27, 1024, 4096), (33, 2064, 8192), (500, 528, 2064)])
def test_serving_chain(T, d, h):
    s = Serve(T, d, h)
    s.run()
    rp.check(s.S, *rp.norm_sum(s.x, s.res, None), "S")
    ref, tol = rp.norm_forward(s.S, s.gain, s.bias, 1e-5)
    rp.check(s.n, ref["Y"], tol["Y"], "n")
    for x, c, sc in ((s.w1, s.c1, s.s1), (s.w2, s.c2, s.s2), (s.n, s.cn, s.sn), (s.u, s.cu, s.su)):
        want, ws = rp.quant(x)
        assert torch.equal(c, want)
        rp.check(sc, ws, rp.E * ws, "scale")
    rp.check(s.u, *rp.int8(s.cn, s.c1, s.sn, s.s1, s.b1, None, "gelu_tanh", BF16), "u")
    rp.check(s.y, *rp.int8(s.cu, s.c2, s.su, s.s2, None, s.S, "none", BF16), "y")


def test_serving_chain_captured():
    s, t = Serve(5, 1024, 4096, seed=2), Serve(5, 1024, 4096, seed=2)
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    gen = torch.Generator("cuda").manual_seed(4)
    for _ in range(4):
        x = torch.randn(s.x.shape, generator=gen, device="cuda")
        s.x.copy_(x)
        t.x.copy_(x)
        t.run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.y, t.y) and torch.equal(s.cu, t.cu)

"""The query/key norm with rotation and the gradient clipping against their definitions in 64 bits,
on the GPU: head layouts, element types, partial and odd rotations, far positions, strides, in place,
empty sizes; tensors of every length and address, mixed types, not finite values."""
from __future__ import annotations

import math

import pytest
import torch

from tests import block_parity as bp

pytestmark = pytest.mark.gpu

block = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.block")
ge = pytest.importorskip("gemm_epilogue_transformer_tiled_amd")

BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


class QK:
    def __init__(self, T, hq, hk, D, rot=None, pairs="half", norm=True, dtype=BF16, far=0, amplitude=1.0, pos=torch.int64,
                 eps=1e-6, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed + T + 7 * D)
        r = lambda *s, std=1.0: (torch.randn(s, generator=gen, device="cuda") * std).to(dtype)  # noqa: E731
        self.T, self.hq, self.hk, self.D, self.rot = T, hq, hk, D, D if rot is None else rot
        self.pairs, self.norm, self.dtype, self.eps, self.amplitude = pairs, norm, dtype, eps, amplitude
        self.q, self.k = r(T, hq, D), r(T, hk, D)
        self.doq, self.dok = r(T, hq, D, std=0.1), r(T, hk, D, std=0.1)
        self.gq, self.gk = (r(D), r(D)) if norm else (None, None)
        self.pos = torch.randint(0, far + 1, (T,), generator=gen, device="cuda").to(pos) + torch.arange(T, device="cuda", dtype=pos)
        self.inv = block.rotary_frequencies(self.rot)[0].cuda()

    def plan(self, **kw):
        return block.QKRotary(self.T, self.hq, self.hk, self.D, rot_dim=self.rot, pairs=self.pairs, norm=self.norm,
                              eps=self.eps, dtype=self.dtype, positions_dtype=self.pos.dtype, **kw)

    def common(self):
        return dict(positions=self.pos, inv_freq=self.inv, amplitude=self.amplitude, gain_q=self.gq, gain_k=self.gk)

    def forward(self, plan=None):
        q, k = torch.full_like(self.q, math.nan), torch.full_like(self.k, math.nan)
        (plan or self.plan()).forward(block.make_qk_args(q=self.q, k=self.k, q_out=q, k_out=k, **self.common()))
        return q, k

    def backward(self, plan=None):
        out = dict(dq=torch.full_like(self.q, math.nan), dk=torch.full_like(self.k, math.nan))
        if self.norm:
            out.update(dgain_q=torch.full((self.D,), math.nan, device="cuda"),
                       dgain_k=torch.full((self.D,), math.nan, device="cuda"))
        (plan or self.plan()).backward(block.make_qk_args(q=self.q, k=self.k, dq_out=self.doq, dk_out=self.dok,
                                                          **self.common(), **out))
        return out

    def ref(self, which, backward):
        x, d, g = (self.q, self.doq, self.gq) if which == "q" else (self.k, self.dok, self.gk)
        return bp.qk(x, d if backward else None, g, self.pos, self.inv, self.amplitude, self.rot, self.pairs, self.eps)

    def check_forward(self, out, what=""):
        for w, got in zip("qk", out):
            if got.numel():
                bp.check(got, *self.ref(w, False), f"{what} {w}")

    def check_backward(self, out, what=""):
        for w in "qk":
            dx, tdx, dg, tdg = self.ref(w, True)
            if out["d" + w].numel():
                bp.check(out["d" + w], dx, tdx, f"{what} d{w}")
            if self.norm and (self.hq if w == "q" else self.hk):
                bp.check(out["dgain_" + w], dg, tdg, f"{what} dgain_{w}")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 64), (80, 40), (96, 24), (256, 256), (128, 32), (8, 8), (2, 2),
                                   (20, 10), (36, 34), (512, 512), (64, 0), (72, 20), (192, 128)])
def test_head_sizes(D, rot, pairs, dtype):
    for norm in (True, False):
        c = QK(37, 3, 2, D, rot, pairs, norm, dtype, far=1000)
        c.check_forward(c.forward(), f"norm {norm}")
        c.check_backward(c.backward(), f"norm {norm}")


@pytest.mark.parametrize("T", [1, 2, 5, 63, 1000, 5000])
@pytest.mark.parametrize("hq,hk", [(1, 0), (0, 1), (8, 1), (32, 8), (13, 13)])
def test_tokens_and_heads(T, hq, hk):
    c = QK(T, hq, hk, 64, far=100)
    c.check_forward(c.forward())
    c.check_backward(c.backward())


def test_no_tokens():
    c = QK(0, 4, 2, 64)
    c.forward()
    out = c.backward()
    assert (out["dgain_q"] == 0).all() and (out["dgain_k"] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_far_positions(dtype):
    """Angles of positions up to 2^31 turn as in 64 bits; 32-bit positions the same."""
    c = QK(50, 2, 1, 64, dtype=dtype, far=2 ** 31 - 200, amplitude=1.25)
    c.check_forward(c.forward())
    c.check_backward(c.backward())
    c32 = QK(50, 2, 1, 64, dtype=dtype, far=2 ** 20, pos=torch.int32)
    c32.check_forward(c32.forward())
    before = c32.forward()
    c32.pos = c32.pos.long()
    for a, b in zip(before, c32.forward()):
        assert torch.equal(a, b)
    c32.pos = -c32.pos
    c32.check_forward(c32.forward(), "negative positions")


@pytest.mark.parametrize("scaling", ["linear", "base", "by_parts"])
def test_scaled_frequencies(scaling):
    c = QK(40, 2, 2, 128, far=200000)
    c.inv, c.amplitude = block.rotary_frequencies(128, scaling=scaling, factor=8.0)
    c.inv = c.inv.cuda()
    c.check_forward(c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pairs", ["half", "interleaved"])
def test_packed_projection_in_place(pairs, dtype):
    """Queries, keys and values side by side, turned where they lie; the values stay as they were."""
    c = QK(70, 4, 2, 64, 32, pairs, dtype=dtype)
    want_q, want_k = c.forward()
    packed = torch.randn(70, 8 * 64, device="cuda").to(dtype)
    q, k = packed[:, :256].view(70, 4, 64), packed[:, 256:384].view(70, 2, 64)
    q.copy_(c.q)
    k.copy_(c.k)
    values = packed[:, 384:].clone()
    st = dict(q_strides=q.stride()[:2], k_strides=k.stride()[:2])
    plan = c.plan(q_out_strides=q.stride()[:2], k_out_strides=k.stride()[:2], **st)
    plan.forward(block.make_qk_args(q=q, k=k, q_out=q, k_out=k, **c.common()))
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(packed[:, 384:], values)
    # gradients in place of the outputs' gradients
    want = c.backward()
    dq, dk = c.doq.clone(), c.dok.clone()
    dg = [torch.empty(64, device="cuda") for _ in range(2)]
    c.plan().backward(block.make_qk_args(q=c.q, k=c.k, dq_out=dq, dk_out=dk, dq=dq, dk=dk, dgain_q=dg[0], dgain_k=dg[1],
                                         **c.common()))
    assert torch.equal(dq, want["dq"]) and torch.equal(dk, want["dk"])
    assert torch.equal(dg[0], want["dgain_q"]) and torch.equal(dg[1], want["dgain_k"])


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_head_major_and_odd_strides(dtype):
    c = QK(33, 3, 2, 64, 48, dtype=dtype)
    want = c.forward()
    # [heads][tokens][head_dim], with a pitch that is no multiple of eight and an odd first address
    def place(x, pitch, first):
        flat = torch.full((first + x.shape[1] * x.shape[0] * pitch,), math.nan, device="cuda", dtype=dtype)
        v = flat.as_strided(x.shape, (pitch, x.shape[0] * pitch, 1), first)
        return flat, v
    for pitch, first in ((64, 0), (67, 1), (72, 8)):
        _, q = place(c.q, pitch, first)
        _, k = place(c.k, pitch, first)
        q.copy_(c.q)
        k.copy_(c.k)
        fq, oq = place(c.q, pitch, first)
        fk, ok = place(c.k, pitch, first)
        st = lambda t: t.stride()[:2]  # noqa: E731
        plan = c.plan(q_strides=st(q), k_strides=st(k), q_out_strides=st(oq), k_out_strides=st(ok))
        plan.forward(block.make_qk_args(q=q, k=k, q_out=oq, k_out=ok, **c.common()))
        assert torch.equal(oq, want[0]) and torch.equal(ok, want[1]), (pitch, first)
        written = torch.zeros_like(fq, dtype=torch.bool).as_strided(c.q.shape, oq.stride(), first)
        mask = torch.zeros(fq.shape, dtype=torch.bool, device="cuda")
        mask.as_strided(c.q.shape, oq.stride(), first).fill_(True)
        assert written.shape == oq.shape and fq[~mask].isnan().all(), "elements between heads written"


def test_rows_of_zeros_and_not_finite_rows():
    c = QK(9, 2, 1, 64)
    want = c.forward()
    c.q[3] = 0
    c.q[4, 1, 5] = math.nan
    c.q[5, 0, 6] = math.inf
    got = c.forward()
    assert (got[0][3] == 0).all()
    assert got[0][4, 1].isnan().all() and torch.equal(got[0][4, 0], want[0][4, 0])
    rest = [0, 1, 2, 6, 7, 8]
    assert torch.equal(got[0][rest], want[0][rest]) and torch.equal(got[1], want[1])
    b = QK(9, 2, 1, 64)
    b.q[3] = 0                                          # r = 1 / sqrt(eps): the gradient stays finite
    b.check_backward(b.backward())


def test_gradient_matches_differences():
    c = QK(4, 2, 1, 16, 12, dtype=FP32)
    out = c.backward()
    gen = torch.Generator("cuda").manual_seed(3)
    v = torch.randn(c.q.shape, generator=gen, device="cuda", dtype=torch.float64)

    def loss(x):
        o, _ = bp.qk(x, None, c.gq.double(), c.pos, c.inv, 1.0, c.rot, c.pairs, c.eps)
        return float((o * c.doq.double()).sum())
    step = 1e-5
    slope = (loss(c.q.double() + step * v) - loss(c.q.double() - step * v)) / (2 * step)
    _, tol, _, _ = c.ref("q", True)
    assert abs(float((out["dq"].double() * v).sum()) - slope) <= float((tol * v.abs()).sum()) + 1e-7


def test_qk_captured_and_replayed():
    c = QK(300, 8, 2, 128)
    plan = c.plan()
    q, k = torch.empty_like(c.q), torch.empty_like(c.k)
    out = dict(dq=torch.empty_like(c.q), dk=torch.empty_like(c.k), dgain_q=torch.empty(128, device="cuda"),
               dgain_k=torch.empty(128, device="cuda"))
    fa = block.make_qk_args(q=c.q, k=c.k, q_out=q, k_out=k, **c.common())
    ba = block.make_qk_args(q=c.q, k=c.k, dq_out=c.doq, dk_out=c.dok, **c.common(), **out)
    plan.forward(fa)
    plan.backward(ba)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(fa)
        plan.backward(ba)
    gen = torch.Generator("cuda").manual_seed(1)
    for _ in range(3):
        c.q.copy_(torch.randn(c.q.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q, k, *out.values())]
        want = [*c.forward(), *c.backward().values()]
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_qk_refusals_on_the_device():
    c = QK(10, 2, 1, 64)
    plan = c.plan()
    q, k = torch.empty_like(c.q), torch.empty_like(c.k)
    for bad in (dict(q_out=None), dict(q=c.q.float()), dict(positions=c.pos.int()), dict(positions=c.pos.cpu()),
                dict(gain_q=None), dict(inv_freq=c.inv[:-1]), dict(q_out=torch.empty(10, 2, 65, device="cuda", dtype=BF16)[..., :64])):
        with pytest.raises(ValueError):
            plan.forward(block.make_qk_args(**{**dict(q=c.q, k=c.k, q_out=q, k_out=k, **c.common()), **bad}))
    # an output laid over another tensor's elements, shifted
    buf = torch.zeros(10 * 128 + 64, device="cuda", dtype=BF16)
    with pytest.raises(ge.GemmEpilogueError):
        plan.forward(block.make_qk_args(q=buf[:1280].view(10, 2, 64), k=c.k, q_out=buf[64:].view(10, 2, 64), k_out=k,
                                        **c.common()))
    torch.cuda.synchronize()


# ---- clipping ----

def clip_case(sizes, seed=0, std=1.0, shift=True):
    """Tensors of the given (length, type), packed without padding, and a copy of each."""
    gen = torch.Generator("cuda").manual_seed(seed)
    flats = {t: torch.randn(sum(n for n, x in sizes if x == t) + 1, generator=gen, device="cuda").mul_(std).to(t)
             for t in (BF16, FP32)}
    at = {BF16: int(shift), FP32: int(shift)}
    got = []
    for n, t in sizes:
        got.append(flats[t][at[t]:at[t] + n])
        at[t] += n
    return got, flats


def exact_norm(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def check_clipped(grads, outs, norm, max_norm, eps):
    want = exact_norm(grads)
    assert abs(float(norm) - want) <= want * (bp.E * 1.001 + 1e-12) + 1e-45
    f = min(1.0, max_norm / (want + eps))
    for i, (g, o) in enumerate(zip(grads, outs)):
        v = g.double() * f
        # the factor and the product in fp32 (3 E covers both), one rounding to the type
        bp.check(o, v, v.abs() * (bp.half_step(g.dtype) + 4 * bp.E) + (2.0 ** -133 if g.dtype == BF16 else 2.0 ** -149), f"tensor {i}")


SIZES = {
    "one": [(1, BF16)],
    "tiny": [(1, FP32), (2, BF16), (3, FP32), (7, BF16), (0, BF16), (9, FP32), (0, FP32)],
    "edges": [(n, t) for n in (15, 16, 17, 255, 2047, 2048, 16383, 16384, 16385, 40000) for t in (BF16, FP32)],
    "many": [(1 + (37 * i) % 500, BF16 if i % 3 else FP32) for i in range(700)],
    "large": [(30_000_001, BF16), (5_000_003, FP32), (4096 * 1000, BF16)],
    "none": [],
    "empty": [(0, BF16), (0, FP32)],
}


@pytest.mark.parametrize("max_norm", [1.0, 1e9, 0.0, math.inf])
@pytest.mark.parametrize("which", list(SIZES))
def test_clip(which, max_norm):
    grads, _ = clip_case(SIZES[which])
    plan = block.GradClip(grads, device="cuda")
    norm = torch.full((1,), math.nan, device="cuda")
    outs, flats = clip_case(SIZES[which], seed=1)
    first = [float(flats[t][0]) for t in (BF16, FP32)]
    plan.run(block.make_clip_args(grads, outs, norm=norm, max_norm=max_norm))
    check_clipped(grads, outs, norm, max_norm, 1e-6)
    assert [float(flats[t][0]) for t in (BF16, FP32)] == first, "written before the first tensor"
    again = torch.full((1,), math.nan, device="cuda")
    plan.run(block.make_clip_args(grads, norm=again, max_norm=max_norm))
    assert torch.equal(again, norm)
    # in place gives the same bits
    plan.run(block.make_clip_args(grads, grads, max_norm=max_norm))
    for a, b in zip(grads, outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("value", [1e30, 1e-30, 3e38, 1e-42])
def test_clip_range(value):
    grads = [torch.full((1000,), value, device="cuda"), torch.full((77,), -value, device="cuda")]
    norm = torch.empty(1, device="cuda")
    outs = [torch.empty_like(g) for g in grads]
    block.GradClip(grads).run(block.make_clip_args(grads, outs, norm=norm, max_norm=1.0, eps=0.0))
    want = exact_norm(grads)
    if want > 3.4e38:
        assert float(norm) == math.inf
    else:
        assert abs(float(norm) - want) <= want * bp.E * 1.001 + 1e-45
    v = grads[0].double() * min(1.0, 1.0 / want)
    assert float((outs[0].double() - v).abs().max()) <= float(v.max()) * 4 * bp.E + 2.0 ** -149


def test_clip_not_finite():
    grads = [torch.ones(100, device="cuda", dtype=BF16), torch.ones(50, device="cuda")]
    norm = torch.empty(1, device="cuda")
    outs = [torch.empty_like(g) for g in grads]
    plan = block.GradClip(grads)
    grads[1][7] = math.inf
    plan.run(block.make_clip_args(grads, outs, norm=norm))
    assert float(norm) == math.inf and (outs[0] == 0).all() and outs[1][7].isnan() and float(outs[1].nansum()) == 0
    grads[0][3] = math.nan
    plan.run(block.make_clip_args(grads, outs, norm=norm))
    assert norm.isnan().all() and all(o.isnan().all() for o in outs)


def test_clip_zero_gradients():
    grads = [torch.zeros(1000, device="cuda", dtype=BF16)]
    norm = torch.empty(1, device="cuda")
    for eps in (1e-6, 0.0):
        outs = [torch.full_like(grads[0], 3.0)]
        block.GradClip(grads).run(block.make_clip_args(grads, outs, norm=norm, max_norm=1.0, eps=eps))
        assert float(norm) == 0 and (outs[0] == 0).all()


def test_clip_refusals_on_the_device():
    grads, _ = clip_case(SIZES["tiny"])
    plan = block.GradClip(grads)
    outs = [torch.empty_like(g) for g in grads]
    norm = torch.empty(1, device="cuda")
    with pytest.raises(ge.GemmEpilogueError):          # the same output twice
        plan2 = block.GradClip([grads[1], grads[1]])
        plan2.run(block.make_clip_args([grads[1], grads[1]], [outs[1], outs[1]], norm=norm))
    with pytest.raises(ge.GemmEpilogueError):          # the same tensor twice, in place
        plan2.run(block.make_clip_args([grads[1], grads[1]], [grads[1], grads[1]], norm=norm))
    plan2.run(block.make_clip_args([grads[1], grads[1]], norm=norm))       # its norm is well defined
    long = torch.randn(100, device="cuda")
    two = block.GradClip([long[:50], long[50:]])
    with pytest.raises(ge.GemmEpilogueError):          # an output over another input
        two.run(block.make_clip_args([long[:50], long[50:]], [long[50:], torch.empty(50, device="cuda")], norm=norm))
    for bad in (dict(max_norm=-1.0), dict(max_norm=math.nan), dict(eps=-1.0), dict(eps=math.nan)):
        with pytest.raises(ge.GemmEpilogueError):
            plan.run(block.make_clip_args(grads, outs, norm=norm, **bad))
    for bad in (dict(grads=grads[:-1], outs=outs[:-1]), dict(grads=grads, outs=None, norm=None),
                dict(grads=[g.double() for g in grads], outs=outs)):
        with pytest.raises(ValueError):
            plan.run(block.make_clip_args(**{**dict(norm=norm), **bad}))
    with pytest.raises(ValueError):
        block.GradClip([torch.ones(4, device="cuda", dtype=torch.float16)])
    torch.cuda.synchronize()


def test_clip_captured_and_replayed():
    grads, flats = clip_case(SIZES["edges"])
    plan = block.GradClip(grads)
    norm = torch.empty(1, device="cuda")
    outs = [torch.empty_like(g) for g in grads]
    args = block.make_clip_args(grads, outs, norm=norm)
    plan.run(args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run(args)
    gen = torch.Generator("cuda").manual_seed(5)
    for turn in range(3):
        for f in flats.values():
            f.copy_(torch.randn(f.shape, generator=gen, device="cuda") * (0.001 if turn == 1 else 1.0))
        graph.replay()
        torch.cuda.synchronize()
        check_clipped(grads, outs, norm, 1.0, 1e-6)
        want = norm.clone()
        plan.run(args)
        assert torch.equal(norm, want)

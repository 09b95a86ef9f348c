"""The gated feed-forward block's kernels against its definition in 64 bits, on the GPU.

Every product form (weights [in][out] and [out][in], every output tile, every activation) at sizes
around the tiles' edges; padded leading dimensions whose padding holds NaN; empty sizes; equal bits
from every tile (they sum in the same order, through different pipelines); streams and graphs."""
from __future__ import annotations

import pytest
import torch

from tests import block_parity as bp

pytestmark = pytest.mark.gpu

block = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.block")
ge = pytest.importorskip("gemm_epilogue_transformer_tiled_amd")

TILES = (block.GE_FFN_TILE_256, block.GE_FFN_TILE_128, block.GE_FFN_TILE_64)
NAN_BITS = 0x7FC0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def normal(gen, shape, std=1.0, pad=0):
    """bf16 normals; with pad, rows pad elements longer whose padding is NaN."""
    t = torch.randn(shape, generator=gen, device="cuda") * std
    if not pad:
        return t.bfloat16()
    full = torch.full((shape[0], shape[1] + pad), float("nan"), device="cuda", dtype=torch.bfloat16)
    full[:, :shape[1]] = t.bfloat16()
    return full[:, :shape[1]]


def blank(shape, pad=0):
    """An output tensor of NaN (a value left over would show)."""
    return torch.full((shape[0], shape[1] + pad), float("nan"), device="cuda", dtype=torch.bfloat16)[:, :shape[1]]


class Case:
    def __init__(self, M, d, h, act="silu", layout="kn", seed=0, pad=0, residual=True):
        gen = torch.Generator("cuda").manual_seed(1000 * M + 10 * d + h + seed)
        wi, wo = ((d, h), (h, d)) if layout == "kn" else ((h, d), (d, h))
        self.M, self.d, self.h, self.act, self.layout, self.pad = M, d, h, act, layout, pad
        p = lambda k: pad * k  # noqa: E731  (paddings of different widths, multiples of 8)
        self.X = normal(gen, (M, d), 1.0, p(1))
        self.Wg, self.Wu = normal(gen, wi, max(d, 1) ** -0.5, p(2)), normal(gen, wi, max(d, 1) ** -0.5, p(2))
        self.Wd = normal(gen, wo, max(h, 1) ** -0.5, p(1))
        self.R = normal(gen, (M, d), 1.0, p(2)) if residual else None
        self.G, self.U = normal(gen, (M, h), 1.5, p(1)), normal(gen, (M, h), 1.0, p(1))
        self.dY = normal(gen, (M, d), 0.1, p(3))
        self.wi, self.wo = wi, wo
        w = lambda shape, k: shape[1] + p(k)  # noqa: E731
        self.ld = dict(ldx=d + p(1), ldy=d + p(4), ldr=d + p(2), ldg=h + p(1), lddy=d + p(3), lddx=d + p(2),
                       ldw=w(wi, 2), ldwd=w(wo, 1), lddw=w(wi, 3), lddwd=w(wo, 2)) if pad else {}

    def plan(self, tile=None, save=True):
        return block.GatedFFN(self.M, self.d, self.h, act=self.act, w_layout=self.layout, residual=self.R is not None,
                              save=save, tile=tile, **self.ld)

    def forward(self, plan=None, tile=None, save=True, stream=None):
        plan = plan or self.plan(tile, save)
        out = {"Y": blank((self.M, self.d), 4 * self.pad)}
        if save:
            out.update(G=blank((self.M, self.h), self.pad), U=blank((self.M, self.h), self.pad))
        plan.forward(block.make_ffn_args(X=self.X, Wg=self.Wg, Wu=self.Wu, Wd=self.Wd, residual=self.R, **out), stream)
        return out

    def backward(self, plan=None, tile=None, dx=True, dw=True, stream=None):
        plan = plan or self.plan(tile)
        out = {"dX": blank((self.M, self.d), 2 * self.pad)} if dx else {}
        if dw:
            out.update(dWg=blank(self.wi, 3 * self.pad), dWu=blank(self.wi, 3 * self.pad), dWd=blank(self.wo, 2 * self.pad))
        plan.backward(block.make_ffn_args(X=self.X, Wg=self.Wg, Wu=self.Wu, Wd=self.Wd, G=self.G, U=self.U, dY=self.dY,
                                          **out), stream)
        return out

    def check_forward(self, out, what):
        ref, tol = bp.ffn_forward(self.X, self.Wg, self.Wu, self.Wd, self.act, self.layout, self.R)
        for k, v in out.items():
            bp.check(v, ref[k], tol[k], f"{what} {k}")

    def check_backward(self, out, what):
        ref, tol = bp.ffn_backward(self.X, self.Wg, self.Wu, self.Wd, self.G, self.U, self.dY, self.act, self.layout)
        for k, v in out.items():
            bp.check(v, ref[k], tol[k], f"{what} {k}")


SIZES = [(1, 8, 8), (2, 64, 128), (7, 136, 72), (16, 256, 264), (33, 64, 520), (64, 64, 64), (65, 72, 136),
         (130, 200, 264), (257, 264, 520), (300, 576, 1032)]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,d,h", SIZES)
def test_forward_sizes(M, d, h, layout):
    c = Case(M, d, h, layout=layout)
    c.check_forward(c.forward(), "auto")
    for tile in TILES:
        c.check_forward(c.forward(tile=tile), f"tile {tile}")


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,d,h", SIZES)
def test_backward_sizes(M, d, h, layout):
    c = Case(M, d, h, layout=layout)
    c.check_backward(c.backward(), "auto")
    for tile in TILES:
        c.check_backward(c.backward(tile=tile), f"tile {tile}")


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh", "silu"])
def test_activations(act, layout):
    c = Case(100, 192, 328, act=act, layout=layout, residual=False)
    for tile in TILES:
        c.check_forward(c.forward(tile=tile), f"{act} tile {tile}")
        c.check_backward(c.backward(tile=tile), f"{act} tile {tile}")
    few = Case(5, 192, 328, act=act, layout=layout)
    few.check_forward(few.forward(save=False), f"{act} few rows")
    few.check_forward(few.forward(), f"{act} few rows, kept")


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M", [3, 150])
def test_padded_rows_are_neither_read_nor_written(M, layout):
    c = Case(M, 136, 264, layout=layout, pad=8)
    for tile in (None, *TILES):
        for out in (c.forward(tile=tile), c.backward(tile=tile)):
            (c.check_forward if "Y" in out else c.check_backward)(out, f"tile {tile}")
            for k, v in out.items():
                rest = v._base[:, v.shape[1]:].view(torch.int16)
                assert (rest == NAN_BITS).all(), f"{k}: padding written"


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_tiles_give_equal_bits(layout):
    c = Case(700, 1096, 1544, layout=layout)
    runs = [{**c.forward(tile=t), **{k: v for k, v in c.backward(tile=t).items()}} for t in TILES]
    for other in runs[1:]:
        for k in runs[0]:
            assert torch.equal(runs[0][k], other[k]), k
    again = {**c.forward(tile=TILES[0]), **c.backward(tile=TILES[0])}
    for k in again:
        assert torch.equal(runs[0][k], again[k]), f"{k}: a second run differs"


@pytest.mark.parametrize("M,d,h", [(2048, 1024, 2816), (1500, 1032, 2856)])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_many_tiles(M, d, h, layout):
    """Several rounds of the largest tile on every compute unit, each race a chance to show."""
    c = Case(M, d, h, layout=layout)
    c.check_forward(c.forward(), "auto")
    c.check_backward(c.backward(), "auto")
    f, b = c.forward(tile=block.GE_FFN_TILE_256), c.backward(tile=block.GE_FFN_TILE_256)
    c.check_forward(f, "forward")
    c.check_backward(b, "backward")
    small = {**c.forward(tile=block.GE_FFN_TILE_64), **c.backward(tile=block.GE_FFN_TILE_64)}
    for k, v in {**f, **b}.items():
        assert torch.equal(v, small[k]), k


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,d,h", [(64, 264, 4104), (40, 2056, 264), (96, 4104, 520), (4100, 72, 136), (130, 1032, 3080),
                                   (20, 520, 4104), (9, 4104, 136)])
def test_split_contractions(M, d, h, layout):
    """Long contractions over few tiles are split over workgroups; the sums meet in one order, so
    that runs agree bit for bit, also when the workspace holds another call's remains."""
    c = Case(M, d, h, layout=layout)
    plan = c.plan()
    first = {**c.forward(plan=plan), **c.backward(plan=plan)}
    c.check_forward({k: first[k] for k in ("Y", "G", "U")}, plan.describe())
    c.check_backward({k: first[k] for k in ("dX", "dWg", "dWu", "dWd")}, plan.describe())
    for _ in range(5):
        again = {**c.forward(plan=plan), **c.backward(plan=plan)}
        for k in first:
            assert torch.equal(first[k], again[k]), (k, plan.describe())


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,d,h", [(1, 2048, 4104), (2, 4104, 2056), (7, 1032, 8200), (15, 2056, 4096), (16, 2184, 4136),
                                   (16, 8200, 1032)])
def test_few_rows_of_large_weights(M, d, h, layout):
    """The kernels that stream the weights through registers, with every edge: rows, columns, contraction."""
    for act, save in (("silu", True), ("gelu_tanh", False), ("relu", True), ("none", False)):
        c = Case(M, d, h, layout=layout, act=act, residual=save)
        plan = c.plan(save=save)
        assert plan.describe().startswith("few rows")
        out = c.forward(plan=plan, save=save)
        c.check_forward(out, act)
        again = c.forward(plan=plan, save=save)
        for k in out:
            assert torch.equal(out[k], again[k]), k
    c.check_backward(c.backward(), "backward")
    c = Case(M, d, h, layout=layout, pad=8)
    out = c.forward()
    c.check_forward(out, "padded")
    for k, v in out.items():
        assert (v._base[:, v.shape[1]:].view(torch.int16) == NAN_BITS).all(), k


def test_splits_are_chosen():
    """The sizes above reach the split kernels of every product (one at least each)."""
    seen = [Case(*s).plan().describe() for s in ((64, 264, 4104), (40, 2056, 264), (96, 4104, 520), (4100, 72, 136))]
    for name in ("pair", "down", "grad", "dx", "dw"):
        assert any(int(w.split("/")[1]) > 1 for line in seen for w in line.split() if w.startswith(name + "=")), (name, seen)


def test_empty_sizes():
    for M, d, h in ((0, 64, 64), (5, 64, 0), (5, 0, 64), (0, 0, 0)):
        c = Case(M, d, h)
        f = c.forward()
        if h == 0:
            assert torch.equal(f["Y"], c.R)
        if d == 0:
            assert (f["G"] == 0).all() and (f["U"] == 0).all()
        b = c.backward()
        for k, v in b.items():
            assert (v == 0).all(), (M, d, h, k)


def test_output_over_the_residual():
    c = Case(77, 128, 264)
    want = c.forward(save=False)["Y"]
    y = c.R.clone()
    c.plan(save=False).forward(block.make_ffn_args(X=c.X, Wg=c.Wg, Wu=c.Wu, Wd=c.Wd, residual=y, Y=y))
    assert torch.equal(y, want)


def test_gradients_left_out():
    c = Case(90, 136, 264)
    whole = c.backward()
    dx, dw = c.backward(dw=False), c.backward(dx=False)
    for part in (dx, dw):
        for k, v in part.items():
            assert torch.equal(v, whole[k]), k


def test_rows_do_not_mix():
    """NaN and infinities in one row reach that row's outputs only."""
    c = Case(130, 136, 264)
    want = c.forward()
    c.X[17, 5], c.X[18, 7] = float("nan"), float("inf")
    got = c.forward()
    rest = [r for r in range(c.M) if r not in (17, 18)]
    for k in got:
        assert torch.equal(got[k][rest], want[k][rest]), k
    assert got["Y"][17].isnan().all()


def test_large_preactivations():
    """Gates far out: the activations and slopes reach their limits, nothing overflows to NaN."""
    for act in ("silu", "gelu_tanh", "relu"):
        c = Case(70, 64, 136, act=act)
        c.G[:, ::3] = 300.0
        c.G[:, 1::3] = -300.0
        c.G[0, 0], c.G[1, 1] = 2.0 ** 100, -(2.0 ** 100)
        c.G[2, 0], c.G[2, 1] = 0.0, -0.0
        b = c.backward(dw=False)
        c.check_backward(b, act)


def test_gradients_match_differences():
    """The block's gradient against central differences of its 64-bit definition: the loss
    sum(dY * Y) moves with X as dX says."""
    c = Case(6, 64, 136, residual=False)
    ref, _ = bp.ffn_forward(c.X, c.Wg, c.Wu, c.Wd, c.act, c.layout)
    c.G, c.U = ref["G"].bfloat16(), ref["U"].bfloat16()
    dX = c.backward(dw=False)["dX"].double()
    gen = torch.Generator("cuda").manual_seed(4)
    v = torch.randn(c.M, c.d, generator=gen, device="cuda", dtype=torch.float64)
    step = 1e-4

    def loss(x):
        g, u = x @ c.Wg.double(), x @ c.Wu.double()
        return float(((bp.act(c.act, g) * u) @ c.Wd.double() * c.dY.double()).sum())
    x = c.X.double()
    slope = (loss(x + step * v) - loss(x - step * v)) / (2 * step)
    # dX carries roundings of G, U, dG, dU and its own, each at most U relative to sums of size ~1
    _, tol = bp.ffn_backward(c.X, c.Wg, c.Wu, c.Wd, c.G, c.U, c.dY, c.act, c.layout)
    g, u, dh = ref["G"].abs(), ref["U"].abs(), (c.dY.double() @ c.Wd.double().t()).abs()
    # G and U themselves are rounded: slopes of every activation change by less than 1.2 per unit
    kept = dh * (u * (1.2 * bp.U * g) + 1.13 * bp.U * u) @ c.Wg.double().abs().t() + \
        dh * (1.13 * bp.U * g) @ c.Wu.double().abs().t()
    assert abs(float((dX * v).sum()) - slope) <= float(((tol["dX"] + kept) * v.abs()).sum()) + 1e-6


def test_streams_and_workspaces():
    a, b = Case(300, 264, 520, seed=1), Case(300, 264, 520, seed=2)
    want = [c.forward()["Y"] for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    plan = a.plan()
    packs = []
    for c in (a, b):
        out = {"Y": blank((c.M, c.d)), "G": blank((c.M, c.h)), "U": blank((c.M, c.h))}
        ws = torch.zeros(plan.workspace_size(), dtype=torch.uint8, device="cuda")
        packs.append((block.make_ffn_args(X=c.X, Wg=c.Wg, Wu=c.Wu, Wd=c.Wd, residual=c.R, workspace=ws, **out), out))
    torch.cuda.synchronize()
    for _ in range(20):
        for (args, _), s in zip(packs, streams):
            plan.forward(args, s.cuda_stream)
    torch.cuda.synchronize()
    for (_, out), w in zip(packs, want):
        assert torch.equal(out["Y"], w)


@pytest.mark.parametrize("M", [1, 9, 200])
def test_captured_and_replayed(M):
    c = Case(M, 264, 520)
    plan = c.plan()
    fo = {"Y": blank((M, c.d)), "G": blank((M, c.h)), "U": blank((M, c.h))}
    bo = {"dX": blank((M, c.d)), "dWg": blank(c.wi), "dWu": blank(c.wi), "dWd": blank(c.wo)}
    fa = block.make_ffn_args(X=c.X, Wg=c.Wg, Wu=c.Wu, Wd=c.Wd, residual=c.R, **fo)
    ba = block.make_ffn_args(X=c.X, Wg=c.Wg, Wu=c.Wu, Wd=c.Wd, G=c.G, U=c.U, dY=c.dY, **bo)
    plan.forward(fa)
    plan.backward(ba)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(fa)
        plan.backward(ba)
    gen = torch.Generator("cuda").manual_seed(7)
    for turn in range(4):
        c.X.copy_(torch.randn(c.X.shape, generator=gen, device="cuda"))
        for t in (*fo.values(), *bo.values()):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in {**fo, **bo}.items()}
        want = {**c.forward(plan=plan), **c.backward(plan=plan)}
        for k in got:
            assert torch.equal(got[k], want[k]), (turn, k)


def test_refusals_on_the_device():
    c = Case(20, 64, 136)
    plan = c.plan()
    ok = dict(X=c.X, Wg=c.Wg, Wu=c.Wu, Wd=c.Wd, residual=c.R, Y=blank((20, 64)), G=blank((20, 136)), U=blank((20, 136)))
    plan.forward(block.make_ffn_args(**ok))
    for bad in (dict(X=c.X.float()), dict(X=c.X[:19]), dict(Y=None), dict(residual=c.R.cpu()), dict(Wg=c.Wg.t()),
                dict(G=blank((20, 136), 8))):
        with pytest.raises(ValueError):
            plan.forward(block.make_ffn_args(**{**ok, **bad}))
    both = torch.zeros(20, 64, device="cuda", dtype=torch.bfloat16)
    for bad in (dict(Y=c.X), dict(G=both.new_empty(20, 136), U=None)):
        with pytest.raises((ValueError, ge.GemmEpilogueError)):
            plan.forward(block.make_ffn_args(**{**ok, **bad}))
    small = torch.zeros(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(ge.GemmEpilogueError):
        plan.forward(block.make_ffn_args(**ok, workspace=small))
    torch.cuda.synchronize()

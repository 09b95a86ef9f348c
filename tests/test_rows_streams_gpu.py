"""The row operators on streams, in graphs and with shared workspaces, on the GPU."""
from __future__ import annotations

import pytest
import torch

from tests import rows_parity as rp

pytestmark = pytest.mark.gpu

block = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.block")
rows = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.rows")

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(BF16)


def busy():
    """Some tens of milliseconds of work on the current stream, and remains in the memory that the next
    workspaces are taken from."""
    torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(50_000_000)


def code(gen, *shape):
    return torch.randint(-127, 128, shape, generator=gen, device="cuda").to(torch.int8)


class All:
    """Every operator once, on inputs of its own."""

    def __init__(self, seed=0, M=300, d=1032, K=4096, N=264, workspace=None):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.rng = torch.tensor([11, 5], dtype=torch.int64, device="cuda")
        e = lambda *s, t=BF16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        f = torch.float32
        self.X, self.R, self.dY, self.dS = normal(gen, M, d), normal(gen, M, d), normal(gen, M, d), normal(gen, M, d)
        self.gain, self.bias = normal(gen, d), normal(gen, d)
        self.S, self.Y, self.dX, self.dR, self.D, self.dD = (e(M, d) for _ in range(6))
        self.mean, self.rstd, self.dgain, self.dbias = e(M, t=f), e(M, t=f), e(d, t=f), e(d, t=f)
        self.codes, self.scale = e(M, d, t=torch.int8), e(M, t=f)
        self.A, self.B, self.xs, self.ws = code(gen, 40, K), code(gen, N, K), torch.rand(40, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
        self.A1 = self.A[:3].clone()
        self.P, self.P1 = e(40, N), e(3, N)
        self.norm = rows.LayerNorm(M, d, residual=True, dropout=0.2, site=1)
        self.drop = rows.Dropout(M, d, 0.3, site=2)
        self.quant = rows.RowQuant(M, d)
        self.i8, self.i81 = rows.Int8Linear(40, N, K), rows.Int8Linear(3, N, K)
        self.na = rows.make_norm_args(X=self.X, residual=self.R, S=self.S, Y=self.Y, gain=self.gain, bias=self.bias, mean=self.mean,
                                      rstd=self.rstd, rng=self.rng, dY=self.dY, dS=self.dS, dX=self.dX, dR=self.dR,
                                      dgain=self.dgain, dbias=self.dbias, workspace=workspace)
        self.da = rows.make_dropout_args(X=self.X, Y=self.D, dY=self.dY, dX=self.dD, rng=self.rng)
        self.qa = rows.make_quant_args(X=self.Y, codes=self.codes, scale=self.scale)
        self.ia = rows.make_i8_args(X=self.A, W=self.B, x_scale=self.xs, w_scale=self.ws, Y=self.P, workspace=workspace)
        self.ia1 = rows.make_i8_args(X=self.A1, W=self.B, x_scale=self.xs[:3], w_scale=self.ws, Y=self.P1)

    def workspace_bytes(self):
        return max(self.norm._workspace_size(), self.i8._workspace_size())

    def run(self, stream=None):
        s = None if stream is None else stream.cuda_stream
        self.norm.forward(self.na, s)
        self.norm.backward(self.na, s)
        self.drop.forward(self.da, s)
        self.drop.backward(self.da, s)
        self.quant.run(self.qa, s)
        self.i8.run(self.ia, s)
        self.i81.run(self.ia1, s)

    def outputs(self):
        return [self.S, self.Y, self.mean, self.rstd, self.dX, self.dR, self.dgain, self.dbias, self.D, self.dD, self.codes, self.scale,
                self.P, self.P1]

    def result(self):
        torch.cuda.synchronize()
        return [t.clone() for t in self.outputs()]

    def spoil(self):
        for t in self.outputs():
            t.fill_(7)


def same(a, b):
    """Which outputs differ is what a failure shows."""
    return [i for i, (x, y) in enumerate(zip(a, b)) if not torch.equal(x, y)] == []


def test_a_split_product_is_among_them():
    assert "splits=1 " not in All().i8.describe() and "few" in All().i81.describe()


def test_on_a_side_stream_behind_a_busy_one():
    a = All()
    a.run()
    want = a.result()
    a.spoil()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy()
    b = All()                                   # its workspaces are made while the current stream is busy
    b.run(side)
    assert same(b.result(), want)
    with torch.cuda.stream(side):
        a.run()                                 # the current stream
    assert same(a.result(), want)


def test_two_streams_at_once():
    """Two plans with workspaces of their own, calls interleaved."""
    a, b = All(seed=1), All(seed=2)
    a.run()
    b.run()
    wa, wb = a.result(), b.result()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.spoil()
        b.spoil()
        torch.cuda.synchronize()
        for _ in range(3):
            a.run(s)
            b.run(t)
        assert same(a.result(), wa) and same(b.result(), wb)


def test_one_plan_on_two_streams_with_workspaces_of_the_packs():
    first = All(seed=3)
    size = first.workspace_bytes()
    packs = [All(seed=3, workspace=torch.zeros(size, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    first.run()
    want = first.result()
    for p in packs:
        p.norm, p.drop, p.quant, p.i8, p.i81 = first.norm, first.drop, first.quant, first.i8, first.i81
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for p in packs:
            p.spoil()
        torch.cuda.synchronize()
        for _ in range(3):
            for p, s in zip(packs, streams):
                p.run(s)
        for p in packs:
            assert same(p.result(), want)


def test_captured_and_replayed_with_new_numbers():
    """A graph reads the offset when it is replayed: new numbers each time, like the same eager calls."""
    a, b = All(seed=4), All(seed=4)
    a.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.rng[1] += 1
        a.run()
    a.rng.copy_(torch.tensor([11, 5]))
    seen = []
    gen = torch.Generator("cuda").manual_seed(5)
    for _ in range(4):
        x = normal(gen, *a.X.shape)
        for o in (a, b):
            o.X.copy_(x)
            o.spoil()
        b.rng[1] += 1
        b.run()
        graph.replay()
        ra, rb = a.result(), b.result()
        assert same(ra, rb) and int(a.rng[1]) == int(b.rng[1])
        seen.append(ra[8] == 0)
        b.rng[1] += 100                          # eager work between the replays
        b.run()
        b.rng[1] -= 100
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
    f = rp.drop_factors(300, 1032, 0.3, 11, 9, 2).cuda()
    assert torch.equal(seen[-1], (f == 0) | (a.X == 0))


def test_one_workspace_for_these_and_the_block_operators_in_turn():
    gen = torch.Generator("cuda").manual_seed(6)
    M, d, h = 64, 264, 4104
    c = dict(X=normal(gen, M, d), Wg=normal(gen, d, h, std=d ** -0.5), Wu=normal(gen, d, h, std=d ** -0.5),
             Wd=normal(gen, h, d, std=h ** -0.5))
    ffn = block.GatedFFN(M, d, h)
    a = All(seed=7)
    a.run()
    Y = torch.empty_like(c["X"])
    ffn.forward(block.make_ffn_args(**c, Y=Y))
    want, wy = a.result(), Y.clone()
    ws = torch.zeros(max(a.workspace_bytes(), ffn.workspace_size()), dtype=torch.uint8, device="cuda")
    b = All(seed=7, workspace=ws)
    fa = block.make_ffn_args(**c, Y=Y, workspace=ws)
    for _ in range(3):
        b.spoil()
        Y.fill_(7)
        b.i8.run(b.ia)
        ffn.forward(fa)
        b.run()
        ffn.forward(fa)
        b.i8.run(b.ia)
        assert same(b.result(), want) and torch.equal(Y, wy)


def test_packs_of_another_plan():
    """A pack that one plan's call has used, with that plan's workspace, serves another plan of the same kind."""
    a, b = All(seed=8), All(seed=8)
    a.run()
    want = a.result()
    a.spoil()
    a.norm, a.i8 = b.norm, b.i8
    del b
    a.run()
    assert same(a.result(), want)

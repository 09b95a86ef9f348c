"""The block operators' workspaces on streams other than torch's current one, on the GPU: the current
stream is busy while plans are made and called elsewhere."""
from __future__ import annotations

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


def busy():
    """Some tens of milliseconds of work on the current stream, and remains in the memory that the next
    workspaces are taken from."""
    torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(50_000_000)


def ffn_backward(plan, c, stream):
    M, d, h = c["X"].shape[0], c["X"].shape[1], c["G"].shape[1]
    out = dict(dX=c["X"].new_empty(M, d), dWg=c["X"].new_empty(d, h), dWu=c["X"].new_empty(d, h), dWd=c["X"].new_empty(h, d))
    args = block.make_ffn_args(**c, **out)
    torch.cuda.synchronize()
    busy()
    plan.backward(args, stream.cuda_stream)
    stream.synchronize()
    got = {k: v.clone() for k, v in out.items()}
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("M,d,h", [(64, 264, 4104), (96, 4104, 520)])
def test_first_feed_forward_backward_on_a_side_stream(M, d, h):
    gen = torch.Generator("cuda").manual_seed(1)
    c = dict(X=normal(gen, M, d), Wg=normal(gen, d, h, std=d ** -0.5), Wu=normal(gen, d, h, std=d ** -0.5),
             Wd=normal(gen, h, d, std=h ** -0.5), G=normal(gen, M, h), U=normal(gen, M, h), dY=normal(gen, M, d, std=0.1))
    plan = block.GatedFFN(M, d, h)                  # without `save`: the backward workspace is made by its first call
    side = torch.cuda.Stream()
    first = ffn_backward(plan, c, side)
    second = ffn_backward(plan, c, torch.cuda.current_stream())
    for k in first:
        assert torch.equal(first[k], second[k]), k


def test_first_rotation_backward_on_a_side_stream():
    gen = torch.Generator("cuda").manual_seed(2)
    T, hq, hk, D = 2000, 4, 2, 64
    c = dict(q=normal(gen, T, hq, D), k=normal(gen, T, hk, D), dq_out=normal(gen, T, hq, D), dk_out=normal(gen, T, hk, D),
             gain_q=normal(gen, D), gain_k=normal(gen, D), positions=torch.arange(T, device="cuda"),
             inv_freq=block.rotary_frequencies(D)[0].cuda())
    plan = block.QKRotary(T, hq, hk, D)
    runs = []
    for stream in (torch.cuda.Stream(), torch.cuda.current_stream()):
        out = dict(dq=torch.empty_like(c["q"]), dk=torch.empty_like(c["k"]), dgain_q=torch.empty(D, device="cuda"),
                   dgain_k=torch.empty(D, device="cuda"))
        args = block.make_qk_args(**c, **out)
        torch.cuda.synchronize()
        busy()
        plan.backward(args, stream.cuda_stream)
        stream.synchronize()
        runs.append({k: v.clone() for k, v in out.items()})
        torch.cuda.synchronize()
    for k in runs[0]:
        assert torch.equal(runs[0][k], runs[1][k]), k


def test_plans_made_behind_a_busy_stream_are_ready_on_another():
    gen = torch.Generator("cuda").manual_seed(3)
    M, d, h = 64, 264, 4104
    X, Wg, Wu, Wd = normal(gen, M, d), normal(gen, d, h, std=0.05), normal(gen, d, h, std=0.05), normal(gen, h, d, std=0.02)
    grads = [normal(gen, 1000), normal(gen, 40000)]
    side, runs = torch.cuda.Stream(), []
    for stream in (side, torch.cuda.current_stream()):
        Y, norm = torch.empty_like(X), torch.empty(1, device="cuda")
        torch.cuda.synchronize()
        busy()
        plan, clip = block.GatedFFN(M, d, h), block.GradClip(grads)
        plan.forward(block.make_ffn_args(X=X, Wg=Wg, Wu=Wu, Wd=Wd, Y=Y), stream.cuda_stream)
        clip.run(block.make_clip_args(grads, norm=norm), stream.cuda_stream)
        torch.cuda.synchronize()
        runs.append((Y, norm))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_one_workspace_for_all_operators_in_turn():
    """Calls of several plans share one workspace, eagerly and in a graph: what one leaves there is never
    another's ticket."""
    gen = torch.Generator("cuda").manual_seed(4)
    sizes = [(64, 264, 4104), (9, 2048, 4104), (333, 520, 1032)]
    ffns, runs = [], []
    for M, d, h in sizes:
        c = dict(X=normal(gen, M, d), Wg=normal(gen, d, h, std=d ** -0.5), Wu=normal(gen, d, h, std=d ** -0.5),
                 Wd=normal(gen, h, d, std=h ** -0.5), dY=normal(gen, M, d, std=0.1))
        ffns.append((block.GatedFFN(M, d, h, save=True), c))
    T, hq, hk, D = 3000, 8, 2, 64
    qk = block.QKRotary(T, hq, hk, D)
    q, k = normal(gen, T, hq, D), normal(gen, T, hk, D)
    heads = dict(q=q, k=k, dq_out=normal(gen, T, hq, D), dk_out=normal(gen, T, hk, D), gain_q=normal(gen, D), gain_k=normal(gen, D),
                 positions=torch.arange(T, device="cuda"), inv_freq=block.rotary_frequencies(D)[0].cuda())
    grads = [normal(gen, 100_000), normal(gen, 3_000_000)]
    clip = block.GradClip(grads)
    e = torch.empty_like
    for shared in (False, True):
        size = max(p.workspace_size(b) for p, _ in ffns for b in (False, True))
        size = max(size, qk.workspace_bytes, clip.workspace.numel())
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda") if shared else None
        outs, calls = [], []
        for plan, c in ffns:
            M, h = c["X"].shape[0], c["Wg"].shape[1]
            o = dict(Y=e(c["X"]), G=c["X"].new_empty(M, h), U=c["X"].new_empty(M, h), dX=e(c["X"]), dWg=e(c["Wg"]),
                     dWu=e(c["Wu"]), dWd=e(c["Wd"]))
            args = block.make_ffn_args(**c, **o, workspace=ws)
            outs += o.values()
            calls += [lambda p=plan, a=args: p.forward(a), lambda p=plan, a=args: p.backward(a)]
        o = dict(dq=e(q), dk=e(k), dgain_q=torch.empty(D, device="cuda"), dgain_k=torch.empty(D, device="cuda"))
        qa = block.make_qk_args(**heads, **o, workspace=ws)
        clipped, norm = [e(g) for g in grads], torch.empty(1, device="cuda")
        ca = block.make_clip_args(grads, clipped, norm=norm, workspace=ws)
        outs += [*o.values(), *clipped, norm]
        others = [lambda: qk.backward(qa), lambda: clip.run(ca)]

        def step():
            for call in calls:
                call()
                for other in others:
                    other()
        step()
        torch.cuda.synchronize()
        runs.append([t.clone() for t in outs])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(2):
            for t in outs:
                t.fill_(float("nan"))
            graph.replay()
            step() if shared else None
            torch.cuda.synchronize()
            runs.append([t.clone() for t in outs])
    for run in runs[1:]:
        for a, b in zip(runs[0], run):
            assert torch.equal(a, b)

"""Host logic of block.py's plans on the CPU, with stand-ins for the library and for torch's streams: on
which stream a workspace is made, and what is refused before anything is launched."""
from __future__ import annotations

import contextlib
import math
import types

import pytest
import torch

import gemm_epilogue_transformer_tiled_amd as ge
from gemm_epilogue_transformer_tiled_amd import block

CURRENT, SIDE = 0x77, 0x1234
BF16 = torch.bfloat16


class World:
    """What happened, in order, and the stream that was current."""

    def __init__(self):
        self.now, self.events, self.capturing = CURRENT, [], ()

    @contextlib.contextmanager
    def on(self, handle):
        before, self.now = self.now, handle
        try:
            yield
        finally:
            self.now = before


@pytest.fixture
def world(monkeypatch):
    w = World()

    def create(*args):
        return ge.GE_OK                    # (no handle: nothing for the real library to destroy)

    def size(*args):
        args[-1]._obj.value = 64
        return ge.GE_OK

    def call(name):
        def f(handle, args, stream):
            w.events.append((name, stream))
            return ge.GE_OK
        return f
    lib = types.SimpleNamespace()
    for name in block.EXPORTED:
        kind = name.split("_", 2)[2]
        setattr(lib, name, create if kind == "create" else size if kind == "workspace_size" else
                (lambda handle: None) if kind == "destroy" else call(name))
    monkeypatch.setattr(block, "lib", lib)
    monkeypatch.setattr(block, "_raw_stream", lambda index: w.now)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
    monkeypatch.setattr(torch.cuda, "stream", lambda handle: w.on(handle))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.now in w.capturing)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(
        cuda_stream=w.now, synchronize=lambda: w.events.append(("waited", w.now))))
    zeros = torch.zeros

    def recorded(*args, **kw):
        w.events.append(("cleared", w.now))
        return zeros(*args, **kw)
    monkeypatch.setattr(torch, "zeros", recorded)
    return w


def t(*shape, dtype=BF16):
    return torch.ones(shape, dtype=dtype)


def ffn_pack(**kw):
    M, d, h = 4, 8, 16
    base = dict(X=t(M, d), Wg=t(d, h), Wu=t(d, h), Wd=t(h, d), Y=t(M, d), G=t(M, h), U=t(M, h), dY=t(M, d), dX=t(M, d),
                dWg=t(d, h), dWu=t(d, h), dWd=t(h, d))
    return block.make_ffn_args(**{**base, **kw})


def qk_pack(heads_q=2, heads_k=1, **kw):
    T, D = 3, 8
    base = dict(q=t(T, heads_q, D), k=t(T, heads_k, D), q_out=t(T, heads_q, D), k_out=t(T, heads_k, D),
                positions=torch.arange(T), inv_freq=t(D // 2, dtype=torch.float32), gain_q=t(D), gain_k=t(D),
                dq_out=t(T, heads_q, D), dk_out=t(T, heads_k, D), dq=t(T, heads_q, D), dk=t(T, heads_k, D),
                dgain_q=t(D, dtype=torch.float32), dgain_k=t(D, dtype=torch.float32))
    return block.make_qk_args(**{**base, **kw})


def ffn():
    return block.GatedFFN(4, 8, 16, device="cpu"), ffn_pack(), "ge_ffn_backward"


def qk():
    return block.QKRotary(3, 2, 1, 8, device="cpu"), qk_pack(), "ge_qk_backward"


@pytest.mark.parametrize("make", [ffn, qk])
@pytest.mark.parametrize("stream", [SIDE, 0, None])
def test_a_workspace_made_by_a_call_is_cleared_on_its_stream(world, make, stream):
    plan, args, name = make()
    world.events.clear()
    plan.backward(args, stream)
    on = CURRENT if stream is None else stream
    assert world.events == [("cleared", on), (name, on)]
    world.events.clear()
    plan.backward(args, stream)
    assert world.events == [(name, on)]


@pytest.mark.parametrize("make", [ffn, qk])
def test_no_workspace_is_made_on_a_capturing_stream(world, make):
    plan, args, _ = make()
    world.capturing = (SIDE,)
    with pytest.raises(RuntimeError):
        plan.backward(args, SIDE)
    plan.backward(args)                    # another stream's capture does not concern it
    plan.backward(args, SIDE)              # made by now


def test_a_plan_waits_for_the_workspace_it_is_made_with(world):
    """The first call may be on any stream."""
    block.GatedFFN(4, 8, 16, device="cpu")
    block.GradClip([t(5)], device="cpu")
    assert world.events == [("cleared", CURRENT), ("waited", CURRENT)] * 2


def clip():
    grads = [t(5)]
    return block.GradClip(grads, device="cpu"), lambda **kw: block.make_clip_args(grads, grads, **kw), \
        lambda plan, args: plan.run(args)


WITH_WORKSPACE = {
    "ffn forward": lambda: (ffn()[0], ffn_pack, lambda plan, args: plan.forward(args)),
    "ffn backward": lambda: (ffn()[0], ffn_pack, lambda plan, args: plan.backward(args)),
    "qk backward": lambda: (qk()[0], qk_pack, lambda plan, args: plan.backward(args)),
    "clip": clip,
}


@pytest.mark.parametrize("which", list(WITH_WORKSPACE))
def test_workspaces_of_another_device_or_not_dense_are_refused(world, which):
    plan, pack, call = WITH_WORKSPACE[which]()
    call(plan, pack(workspace=torch.empty(256, dtype=torch.uint8)))
    world.events.clear()
    for bad in (torch.empty(256, dtype=torch.uint8, device="meta"), torch.empty(512, dtype=torch.uint8)[::2],
                torch.empty(1, dtype=torch.uint8).expand(256)):
        with pytest.raises(ValueError, match="workspace"):
            call(plan, pack(workspace=bad))
    assert world.events == []              # nothing was launched


@pytest.mark.parametrize("heads_q,heads_k,name", [(2, 0, "dgain_k"), (0, 2, "dgain_q")])
def test_gain_gradients_of_a_side_without_heads(world, heads_q, heads_k, name):
    """They may be left out; one that is given is written (zeros), so it has to fit."""
    plan = block.QKRotary(3, heads_q, heads_k, 8, device="cpu")
    plan.backward(qk_pack(heads_q, heads_k, **{name: None}))
    plan.backward(qk_pack(heads_q, heads_k))
    world.events.clear()
    for bad in (t(4, dtype=torch.float32), t(8), t(16, dtype=torch.float32)[::2], torch.empty(8, device="meta")):
        with pytest.raises(ValueError, match=name):
            plan.backward(qk_pack(heads_q, heads_k, **{name: bad}))
    assert world.events == []


@pytest.mark.parametrize("q_strides", [(0, 0), (0, 8), (8, 0), (16, 4)])
def test_repeated_inputs_have_packed_gradients(world, q_strides):
    """Inputs may repeat, their gradients may not: unless strides are given for these, they are packed."""
    plan = block.QKRotary(3, 2, 1, 8, q_strides=q_strides, device="cpu")
    d = plan.desc
    assert (d.q_token, d.q_head) == q_strides and (d.dq_token, d.dq_head) == (16, 8)
    assert plan.strides["dq"] == (16, 8) and plan.strides["dk"] == (8, 8)


def test_gradients_follow_inputs_that_keep_heads_apart(world):
    for strides in ((16, 8), (64, 8), (8, 24), (64, 16)):
        plan = block.QKRotary(3, 2, 1, 8, q_strides=strides, device="cpu")
        assert (plan.desc.dq_token, plan.desc.dq_head) == strides
    one = block.QKRotary(1, 2, 1, 8, q_strides=(0, 8), device="cpu")          # one token: its stride does not matter
    assert one.strides["dq"] == (0, 8)


def test_frequencies_blended_over_no_range():
    """With slow = fast nothing is blended: what makes fewer turns is divided, what makes as many is kept."""
    plain, _ = block.rotary_frequencies(64)
    turns = 4096 * plain.double() / (2 * math.pi)
    for border in (1.0, 7.5, 4096 / (2 * math.pi)):             # (the last: the first frequency's own)
        got, _ = block.rotary_frequencies(64, scaling="by_parts", factor=4.0, slow=border, fast=border)
        kept = turns > border * (1 + 1e-6)
        divided = turns < border * (1 - 1e-6)
        assert torch.equal(got[kept], plain[kept]) and torch.equal(got[divided], plain[divided] / 4)
        assert got.isfinite().all()


@pytest.mark.parametrize("bad", [dict(slow=2.0, fast=1.0), dict(slow=math.nan), dict(original_length=0), dict(base=0.0),
                                 dict(base=-1.0), dict(base=math.inf), dict(base=math.nan)])
def test_frequencies_refused(bad):
    with pytest.raises(ValueError):
        block.rotary_frequencies(64, scaling="by_parts", factor=4.0, **bad)

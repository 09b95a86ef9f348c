"""Host logic of rows.py's plans on the CPU, with stand-ins for the library and for torch's streams: on which
stream a workspace is made, and what is refused before anything is launched."""
from __future__ import annotations

import contextlib
import types

import pytest
import torch

import gemm_epilogue_transformer_tiled_amd as ge
from gemm_epilogue_transformer_tiled_amd import block, rows

CURRENT, SIDE = 0x77, 0x1234
BF16, FP32 = torch.bfloat16, torch.float32


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
            w.events.append((name, stream, getattr(args._obj, "workspace", None) is not None))
            return ge.GE_OK
        return f
    lib = types.SimpleNamespace()
    for name in rows.EXPORTED:
        kind = name.split("_", 2)[2]
        setattr(lib, name, create if kind == "create" else size if kind == "workspace_size" else
                (lambda handle: None) if kind == "destroy" else call(name))
    monkeypatch.setattr(rows, "lib", lib)
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


M, D = 6, 16


def t(*shape, dtype=BF16):
    return torch.ones(shape, dtype=dtype)


def norm_pack(**kw):
    base = dict(X=t(M, D), residual=t(M, D), S=t(M, D), Y=t(M, D), gain=t(D), bias=t(D), mean=t(M, dtype=FP32), rstd=t(M, dtype=FP32),
                rng=t(2, dtype=torch.int64), dY=t(M, D), dS=t(M, D), dX=t(M, D), dR=t(M, D), dgain=t(D, dtype=FP32),
                dbias=t(D, dtype=FP32))
    return rows.make_norm_args(**{**base, **kw})


def norm(**kw):
    return rows.LayerNorm(M, D, residual=True, dropout=0.1, device="cpu", **kw)


def dropout_pack(**kw):
    base = dict(X=t(M, D), residual=t(M, D), Y=t(M, D), dY=t(M, D), dX=t(M, D), rng=t(2, dtype=torch.int64))
    return rows.make_dropout_args(**{**base, **kw})


def dropout(**kw):
    return rows.Dropout(M, D, 0.1, residual=True, device="cpu", **kw)


def quant_pack(**kw):
    base = dict(X=t(M, D), codes=t(M, D, dtype=torch.int8), scale=t(M, dtype=FP32))
    return rows.make_quant_args(**{**base, **kw})


def quant(**kw):
    return rows.RowQuant(M, D, device="cpu", **kw)


def i8_pack(**kw):
    base = dict(X=t(M, D, dtype=torch.int8), W=t(8, D, dtype=torch.int8), x_scale=t(M, dtype=FP32), w_scale=t(8, dtype=FP32),
                bias=t(8), residual=t(M, 8), Y=t(M, 8))
    return rows.make_i8_args(**{**base, **kw})


def i8(**kw):
    return rows.Int8Linear(M, 8, D, bias=True, residual=True, device="cpu", **kw)


@pytest.mark.parametrize("stream", [SIDE, 0, None])
def test_the_gradients_workspace_is_cleared_on_its_calls_stream(world, stream):
    plan, args = norm(), norm_pack()
    plan.forward(args, stream)
    on = CURRENT if stream is None else stream
    assert world.events == [("ge_norm_forward", on, False)]
    world.events.clear()
    plan.backward(args, stream)
    assert world.events == [("cleared", on), ("ge_norm_backward", on, True)]
    world.events.clear()
    plan.backward(args, stream)
    assert world.events == [("ge_norm_backward", on, True)]


def test_gradients_of_the_rows_alone_need_no_workspace(world):
    plan = norm()
    plan.backward(norm_pack(dgain=None, dbias=None))
    assert world.events == [("ge_norm_backward", CURRENT, False)]
    world.capturing = (CURRENT,)
    plan.backward(norm_pack(dgain=None, dbias=None))
    with pytest.raises(RuntimeError):
        plan.backward(norm_pack())
    world.capturing = ()
    plan.backward(norm_pack())
    world.capturing = (CURRENT,)
    plan.backward(norm_pack())                 # made by now


def test_a_plan_waits_for_the_workspace_it_is_made_with(world):
    """The first call may be on any stream."""
    plan = i8()
    assert world.events == [("cleared", CURRENT), ("waited", CURRENT)]
    world.events.clear()
    plan.run(i8_pack(), SIDE)
    assert world.events == [("ge_i8_run", SIDE, True)]


def test_a_packs_own_workspace_is_used(world):
    for plan, pack, call in ((norm(), norm_pack, "backward"), (i8(), i8_pack, "run")):
        ws = torch.ones(256, dtype=torch.uint8)
        args = pack(workspace=ws)
        getattr(plan, call)(args)
        assert args.c.workspace == ws.data_ptr() and args.c.workspace_bytes == 256
        world.events.clear()
        for bad in (torch.empty(256, dtype=torch.uint8, device="meta"), torch.empty(512, dtype=torch.uint8)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                getattr(plan, call)(pack(workspace=bad))
        assert world.events == []              # nothing was launched


CALLS = {
    "norm forward": (norm, norm_pack, "forward", ("X", "residual", "S", "Y", "gain", "bias", "mean", "rstd", "rng"),
                     ("S", "gain", "bias", "mean", "rstd")),
    "norm backward": (norm, norm_pack, "backward", ("dY", "S", "dS", "gain", "mean", "rstd", "rng", "dX", "dR", "dgain", "dbias"),
                      ("dS", "gain", "dX", "dR", "dgain", "dbias")),
    "dropout forward": (dropout, dropout_pack, "forward", ("X", "residual", "Y", "rng"), ()),
    "dropout backward": (dropout, dropout_pack, "backward", ("dY", "dX", "rng"), ()),
    "quant": (quant, quant_pack, "run", ("X", "codes", "scale"), ()),
    "i8": (i8, i8_pack, "run", ("X", "W", "x_scale", "w_scale", "bias", "residual", "Y"), ()),
}


@pytest.mark.parametrize("which", list(CALLS))
def test_tensors_that_do_not_fit_are_refused(world, which):
    make, pack, call, names, optional = CALLS[which]
    plan = make()
    getattr(plan, call)(pack())
    assert sum(e[0].startswith("ge_") for e in world.events) == 1
    world.events.clear()
    for name in names:
        good = pack().tensors[name]
        wrong = [good.to("meta"), good.double(), torch.cat([good, good]), torch.stack([good, good], -1)[..., 0]]
        if good.dim() == 2:
            wrong += [torch.ones(good.shape[0], good.shape[1] + 8).to(good.dtype)[:, :good.shape[1]], good[:, :-1], good[:-1]]
        for bad in wrong:
            with pytest.raises(ValueError, match=name):
                getattr(plan, call)(pack(**{name: bad}))
        if name in optional:
            getattr(plan, call)(pack(**{name: None}))
            world.events.clear()
        else:
            with pytest.raises(ValueError, match=name):
                getattr(plan, call)(pack(**{name: None}))
    assert world.events == []


def test_leading_dimensions(world):
    wide = lambda n, ld, dtype=BF16: torch.ones(M, ld).to(dtype)[:, :n]  # noqa: E731
    rows.LayerNorm(M, D, ldx=24, ldy=40, device="cpu").forward(rows.make_norm_args(X=wide(D, 24), Y=wide(D, 40)))
    rows.Dropout(M, D, 0.5, lddy=17, device="cpu").backward(
        rows.make_dropout_args(dY=wide(D, 17), dX=t(M, D), rng=t(2, dtype=torch.int64)))
    rows.RowQuant(M, D, ldq=20, device="cpu").run(rows.make_quant_args(X=t(M, D), codes=wide(D, 20, torch.int8), scale=t(M, dtype=FP32)))
    plan = rows.Int8Linear(M, 8, D, ldx=32, ldw=48, ldy=24, ldr=16, device="cpu")
    assert (plan.desc.ldx, plan.desc.ldw, plan.desc.ldy, plan.desc.ldr) == (32, 48, 24, 16)
    for make in (lambda: rows.LayerNorm(M, D, ldq=16, device="cpu"), lambda: rows.Dropout(M, D, 0.5, lds=16, device="cpu"),
                 lambda: rows.RowQuant(M, D, ldy=16, device="cpu"), lambda: rows.Int8Linear(M, 8, D, ldq=16, device="cpu")):
        with pytest.raises(TypeError):
            make()


def test_types_and_names(world):
    for make in (lambda: rows.LayerNorm(M, D, dtype=torch.float16, device="cpu"),
                 lambda: rows.Dropout(M, D, 0.5, dtype=torch.float64, device="cpu"),
                 lambda: rows.RowQuant(M, D, dtype=torch.int8, device="cpu"),
                 lambda: rows.Int8Linear(M, 8, D, dtype=torch.float16, device="cpu")):
        with pytest.raises(ValueError):
            make()
    with pytest.raises(KeyError):
        rows.Int8Linear(M, 8, D, act="tanh", device="cpu")


def test_random_numbers_are_asked_for_where_a_mask_is_drawn(world):
    """Not without dropout, nor where p is below half a step of 2^-16, nor for gradients without dX."""
    for p, needed in ((0.0, False), (7e-6, False), (8e-6, True), (0.5, True)):
        plan = rows.LayerNorm(M, D, dropout=p, device="cpu")
        call = lambda: plan.forward(rows.make_norm_args(X=t(M, D), Y=t(M, D)))  # noqa: E731
        if needed:
            with pytest.raises(ValueError, match="rng"):
                call()
        else:
            call()
    norm().backward(norm_pack(dX=None, rng=None))


def test_refusals_without_the_stand_ins(monkeypatch):
    """The real library: refused before a device is asked for."""
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    for make in (lambda: rows.LayerNorm(M, D, dropout=1.0, device="cpu"), lambda: rows.LayerNorm(M, 0, device="cpu"),
                 lambda: rows.LayerNorm(M, 40000, device="cpu"), lambda: rows.Dropout(M, D, -0.1, device="cpu"),
                 lambda: rows.RowQuant(-1, D, device="cpu"), lambda: rows.Int8Linear(M, 12, D, device="cpu"),
                 lambda: rows.Int8Linear(M, 8, 20, device="cpu"), lambda: rows.Int8Linear(M, 8, 1 << 17, device="cpu")):
        with pytest.raises(ge.GemmEpilogueError):
            make()

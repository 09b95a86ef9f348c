"""Binding of libge_rows.so: the operators on the rows between a transformer's products.

Layer norm with dropout and residual add in front of it, and its gradients (``LayerNorm``), dropout from a
counter-based generator (``Dropout``), int8 codes with a scale per row (``RowQuant``) and the product of
int8 codes with scales per token and per channel (``Int8Linear``).  ``lib`` holds the C functions of
``include/ge_rows.h``; plans and packs are used like those of ``block``: a plan owns one handle and its
zero-filled workspace, a pack of tensors is made once and passed to every call on them.

A call may run on any stream of the plan's device; as with tensors used on a stream that is not their own,
a plan is kept until its calls on other streams than the current one have run, and as long as a graph that
holds them.  Calls that share a plan's workspace must be ordered (give concurrent calls, and graphs that
replay at once, packs with workspaces of their own).

Argument marshalling only: every step of the computation runs in the HIP kernels.  The classes check
shapes, strides, element types and devices of the tensors they are given; the library checks pointers and
sizes again.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import ACT_NAMES, GE_OK, GemmEpilogueError
from .block import DTYPES, Args, _Plan, _check

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libge_rows.so")

GE_I8_TILE_256, GE_I8_TILE_128, GE_I8_TILE_64, GE_I8_TILE_COUNT = range(4)

_p, _i32, _i64, _u32, _f, _sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float,
                                 ctypes.c_size_t)


class ge_norm_desc_t(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("rows", "d", "ldx", "ldr", "lds", "ldy", "lddy", "ldds", "lddx", "lddr")] + \
               [("dtype", _i32), ("residual", _i32), ("site", _u32), ("dropout", _f), ("eps", _f)]


class ge_norm_args_t(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("X", "residual", "S", "Y", "gain", "bias", "mean", "rstd", "rng", "dY", "dS", "dX", "dR",
                                  "dgain", "dbias", "workspace")] + [("workspace_bytes", _sz)]


class ge_dropout_desc_t(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("rows", "d", "ldx", "ldr", "ldy", "lddy", "lddx")] + \
               [("dtype", _i32), ("residual", _i32), ("site", _u32), ("p", _f)]


class ge_dropout_args_t(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("X", "residual", "Y", "dY", "dX", "rng")]


class ge_quant_desc_t(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("rows", "d", "ldx", "ldq")] + [("dtype", _i32)]


class ge_quant_args_t(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("X", "codes", "scale")]


class ge_i8_desc_t(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("M", "N", "K", "ldx", "ldw", "ldy", "ldr")] + \
               [(n, _i32) for n in ("act", "bias", "residual", "dtype", "tile")]


class ge_i8_args_t(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("X", "W", "x_scale", "w_scale", "bias", "residual", "Y", "workspace")] + \
               [("workspace_bytes", _sz)]


def _signatures():
    for name, desc, args, runs in (("norm", ge_norm_desc_t, ge_norm_args_t, ("forward", "backward")),
                                   ("dropout", ge_dropout_desc_t, ge_dropout_args_t, ("forward", "backward")),
                                   ("quant", ge_quant_desc_t, ge_quant_args_t, ("run",)),
                                   ("i8", ge_i8_desc_t, ge_i8_args_t, ("run",))):
        yield f"ge_{name}_validate", ([ctypes.POINTER(desc)], ctypes.c_int)
        yield f"ge_{name}_create", ([ctypes.POINTER(desc), ctypes.POINTER(_p)], ctypes.c_int)
        for r in runs:
            yield f"ge_{name}_{r}", ([_p, ctypes.POINTER(args), _p], ctypes.c_int)
        yield f"ge_{name}_destroy", ([_p], None)
    for name in ("norm", "i8"):
        yield f"ge_{name}_workspace_size", ([_p, ctypes.POINTER(_sz)], ctypes.c_int)
    yield "ge_i8_describe", ([_p, ctypes.c_char_p, _sz], ctypes.c_int)


_SIGS = dict(_signatures())
EXPORTED = tuple(_SIGS)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python gemm_epilogue_transformer_tiled_amd/build.py` "
                          "(there is no host fallback for this library)")
    handle = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in _SIGS.items():
        fn = getattr(handle, name)
        fn.argtypes, fn.restype = args, res
    return handle


lib = _load()


class _RowsPlan(_Plan):
    """A plan of this library: ``_kind`` is the operator's part of the C names."""

    _kind = None
    _calls = ("forward", "backward")
    workspace = None             # of plans that need one

    def _make(self) -> None:
        create = getattr(lib, f"ge_{self._kind}_create")
        self._create(lambda out: create(ctypes.byref(self.desc), out), f"ge_{self._kind}_create")
        self._fns = {call: getattr(lib, f"ge_{self._kind}_{call}") for call in self._calls}

    def _workspace_size(self) -> int:
        n = _sz()
        _check(getattr(lib, f"ge_{self._kind}_workspace_size")(self.handle, ctypes.byref(n)), f"ge_{self._kind}_workspace_size")
        return n.value

    def _dtype(self, dtype) -> int:
        if dtype not in DTYPES:
            raise ValueError(f"element type {dtype}: bfloat16 or float32")
        self.dtype = dtype
        return DTYPES[dtype]

    def _rows(self, args: Args, name: str, ld: int, optional: bool = False) -> None:
        self._tensor(args, name, (self.desc.rows, self.desc.d), self.dtype, (ld, 1), optional=optional)

    def _call(self, call: str, args: Args, stream: Optional[int]) -> None:
        """Checks the pack once for this plan and this call, then makes it."""
        stream = self._stream(stream)
        if call not in args._fits.get(self, ()):
            getattr(self, "_fit_" + call)(args, stream)
            args._fits[self] = (*args._fits.get(self, ()), call)
        if self.workspace is not None and args.tensors["workspace"] is None:
            args.c.workspace, args.c.workspace_bytes = self.workspace.data_ptr(), self.workspace.numel()
        st = self._fns[call](self.handle, args._ref, stream)
        if st != GE_OK:
            raise GemmEpilogueError(st, f"ge_{self._kind}_{call}")

    def close(self) -> None:
        if self.handle:
            getattr(lib, f"ge_{self._kind}_destroy")(self.handle)
            self.handle = None


def _pack(struct, tensors) -> Args:
    a = Args(struct, tensors)
    if "workspace" in tensors:
        w = tensors["workspace"]
        a.c.workspace_bytes = 0 if w is None else w.numel() * w.element_size()
    return a


def _pitches(d: int, names, ld) -> dict:
    for name in ld:
        if name not in names:
            raise TypeError(f"unknown leading dimension {name}")
    return {name: ld.get(name, d) for name in names}


def _site(site: int) -> int:
    """The dropout's number in its step (ctypes would keep its low 32 bits: another site's masks)."""
    if not 0 <= site < 1 << 32:
        raise ValueError(f"site {site}: 0 to 2**32 - 1")
    return site


def make_norm_args(X=None, residual=None, S=None, Y=None, gain=None, bias=None, mean=None, rstd=None, rng=None, dY=None, dS=None,
                   dX=None, dR=None, dgain=None, dbias=None, workspace=None) -> Args:
    """Pointer pack of the layer norm: matrices [rows][d], gain, bias [d] of the plan's type (None: ones,
    zeros), mean, rstd [rows] and dgain, dbias [d] float32, rng an int64 tensor of a seed and an offset."""
    return _pack(ge_norm_args_t(), dict(X=X, residual=residual, S=S, Y=Y, gain=gain, bias=bias, mean=mean, rstd=rstd, rng=rng,
                                        dY=dY, dS=dS, dX=dX, dR=dR, dgain=dgain, dbias=dbias, workspace=workspace))


class LayerNorm(_RowsPlan):
    """Layer norm of rows of d values, Y = norm(S) * gain + bias with S = R + drop(X), and its gradients.

    ``forward`` reads X (and, with ``residual``, the tensor of that name), gain, bias and, with dropout, rng;
    writes Y and, where they are given, S, mean and rstd.  ``backward`` reads dY, S (X itself where there is
    neither residual nor dropout), mean, rstd, gain, dS where it is given (the gradient that reaches S
    from elsewhere) and rng; writes dX, dR (the residual's gradient), dgain and dbias, each if given.
    ``site`` (32 bits) tells the dropouts of one step apart.  ``ld``: leading dimensions that differ (ldx, ldr, lds,
    ldy, lddy, ldds, lddx, lddr)."""

    _kind = "norm"

    def __init__(self, rows: int, d: int, eps: float = 1e-5, dtype=torch.bfloat16, residual: bool = False,
                 dropout: float = 0.0, site: int = 0, device="cuda", **ld: int):
        super().__init__(device)
        self.desc = ge_norm_desc_t(rows=rows, d=d, dtype=self._dtype(dtype), residual=int(residual), site=_site(site),
                                   dropout=dropout, eps=eps, **_pitches(d, ("ldx", "ldr", "lds", "ldy", "lddy", "ldds", "lddx", "lddr"), ld))
        self._make()
        self.drops = self.desc.dropout * 65536 >= 0.5
        # (the workspace is made by the first backward that needs it)

    def _vectors(self, args: Args, *names: str) -> None:
        for n in names:
            self._tensor(args, n, (self.desc.d,), self.dtype, (1,), optional=True)

    def _fit_forward(self, args: Args, stream: int) -> None:
        c = self.desc
        self._rows(args, "X", c.ldx)
        if c.residual:
            self._rows(args, "residual", c.ldr)
        self._rows(args, "S", c.lds, optional=True)
        self._rows(args, "Y", c.ldy)
        self._vectors(args, "gain", "bias")
        for n in ("mean", "rstd"):
            self._tensor(args, n, (c.rows,), torch.float32, (1,), optional=True)
        if self.drops and c.rows:
            self._tensor(args, "rng", (2,), torch.int64, (1,))

    def _fit_backward(self, args: Args, stream: int) -> None:
        c = self.desc
        self._rows(args, "dY", c.lddy)
        self._rows(args, "S", c.lds)
        for n, ld in (("dS", c.ldds), ("dX", c.lddx), ("dR", c.lddr)):
            self._rows(args, n, ld, optional=True)
        self._vectors(args, "gain")
        for n in ("mean", "rstd"):
            self._tensor(args, n, (c.rows,), torch.float32, (1,))
        for n in ("dgain", "dbias"):
            self._tensor(args, n, (c.d,), torch.float32, (1,), optional=True)
        if self.drops and c.rows and args.tensors["dX"] is not None:
            self._tensor(args, "rng", (2,), torch.int64, (1,))
        self._workspace(args)
        needed = args.tensors["dgain"] is not None or args.tensors["dbias"] is not None
        if needed and args.tensors["workspace"] is None and self.workspace is None:
            self.workspace = self._scratch(self._workspace_size(), stream)

    def forward(self, args: Args, stream: Optional[int] = None) -> None:
        self._call("forward", args, stream)

    def backward(self, args: Args, stream: Optional[int] = None) -> None:
        self._call("backward", args, stream)


def make_dropout_args(X=None, residual=None, Y=None, dY=None, dX=None, rng=None) -> Args:
    """Pointer pack of the dropout: matrices [rows][d], rng an int64 tensor of a seed and an offset."""
    return _pack(ge_dropout_args_t(), dict(X=X, residual=residual, Y=Y, dY=dY, dX=dX, rng=rng))


class Dropout(_RowsPlan):
    """Dropout of rows of d values: ``forward`` Y = drop(X) (+ R), ``backward`` dX = drop(dY) with the same mask,
    which the numbers in rng, the site and d determine.  ``ld``: leading dimensions that differ (ldx, ldr, ldy,
    lddy, lddx)."""

    _kind = "dropout"

    def __init__(self, rows: int, d: int, p: float, dtype=torch.bfloat16, residual: bool = False, site: int = 0, device="cuda",
                 **ld: int):
        super().__init__(device)
        self.desc = ge_dropout_desc_t(rows=rows, d=d, dtype=self._dtype(dtype), residual=int(residual), site=_site(site), p=p,
                                      **_pitches(d, ("ldx", "ldr", "ldy", "lddy", "lddx"), ld))
        self._make()

    def _fit_rng(self, args: Args) -> None:
        if self.desc.rows and self.desc.d:
            self._tensor(args, "rng", (2,), torch.int64, (1,))

    def _fit_forward(self, args: Args, stream: int) -> None:
        c = self.desc
        self._rows(args, "X", c.ldx)
        if c.residual:
            self._rows(args, "residual", c.ldr)
        self._rows(args, "Y", c.ldy)
        self._fit_rng(args)

    def _fit_backward(self, args: Args, stream: int) -> None:
        self._rows(args, "dY", self.desc.lddy)
        self._rows(args, "dX", self.desc.lddx)
        self._fit_rng(args)

    def forward(self, args: Args, stream: Optional[int] = None) -> None:
        self._call("forward", args, stream)

    def backward(self, args: Args, stream: Optional[int] = None) -> None:
        self._call("backward", args, stream)


def make_quant_args(X=None, codes=None, scale=None) -> Args:
    """Pointer pack of the codes: X [rows][d], codes int8 [rows][d], scale float32 [rows]."""
    return _pack(ge_quant_args_t(), dict(X=X, codes=codes, scale=scale))


class RowQuant(_RowsPlan):
    """int8 codes and a scale for every row (tokens, or the channels of an [out][in] weight): scale =
    max |x| / 127, code = x / scale to the nearest integer.  ``ld``: leading dimensions that differ (ldx, ldq)."""

    _kind = "quant"
    _calls = ("run",)

    def __init__(self, rows: int, d: int, dtype=torch.bfloat16, device="cuda", **ld: int):
        super().__init__(device)
        self.desc = ge_quant_desc_t(rows=rows, d=d, dtype=self._dtype(dtype), **_pitches(d, ("ldx", "ldq"), ld))
        self._make()

    def _fit_run(self, args: Args, stream: int) -> None:
        c = self.desc
        self._rows(args, "X", c.ldx)
        self._tensor(args, "codes", (c.rows, c.d), torch.int8, (c.ldq, 1))
        self._tensor(args, "scale", (c.rows,), torch.float32, (1,))

    def run(self, args: Args, stream: Optional[int] = None) -> None:
        self._call("run", args, stream)


def make_i8_args(X=None, W=None, x_scale=None, w_scale=None, bias=None, residual=None, Y=None, workspace=None) -> Args:
    """Pointer pack of the product of codes: X int8 [M][K], W int8 [N][K], x_scale [M] and w_scale [N] float32,
    bias [N], residual and Y [M][N] of the plan's type."""
    return _pack(ge_i8_args_t(), dict(X=X, W=W, x_scale=x_scale, w_scale=w_scale, bias=bias, residual=residual, Y=Y,
                                      workspace=workspace))


class Int8Linear(_RowsPlan):
    """Product of int8 codes, Y = act(x_scale[m] * w_scale[n] * (X W^T)[m][n] + bias[n]) + R, with exact sums.

    ``dtype``: that of Y, bias and R.  tile: a ge_i8_tile_t (None: chosen by size).  ``ld``: leading dimensions that
    differ (ldx, ldw, ldy, ldr)."""

    _kind = "i8"
    _calls = ("run",)

    def __init__(self, M: int, N: int, K: int, act: str = "none", bias: bool = False, residual: bool = False,
                 dtype=torch.bfloat16, tile: Optional[int] = None, device="cuda", **ld: int):
        super().__init__(device)
        pitch = {**_pitches(K, ("ldx", "ldw"), {k: v for k, v in ld.items() if k in ("ldx", "ldw")}),
                 **_pitches(N, ("ldy", "ldr"), {k: v for k, v in ld.items() if k not in ("ldx", "ldw")})}
        self.desc = ge_i8_desc_t(M=M, N=N, K=K, act=ACT_NAMES[act], bias=int(bias), residual=int(residual),
                                 dtype=self._dtype(dtype), tile=0 if tile is None else tile + 1, **pitch)
        self._make()
        size = self._workspace_size()
        self.workspace = self._scratch(size) if size else None

    def describe(self) -> str:
        buf = ctypes.create_string_buffer(256)
        _check(lib.ge_i8_describe(self.handle, buf, len(buf)), "ge_i8_describe")
        return buf.value.decode()

    def _fit_run(self, args: Args, stream: int) -> None:
        c = self.desc
        self._tensor(args, "X", (c.M, c.K), torch.int8, (c.ldx, 1))
        self._tensor(args, "W", (c.N, c.K), torch.int8, (c.ldw, 1))
        self._tensor(args, "x_scale", (c.M,), torch.float32, (1,))
        self._tensor(args, "w_scale", (c.N,), torch.float32, (1,))
        if c.bias:
            self._tensor(args, "bias", (c.N,), self.dtype, (1,))
        if c.residual:
            self._tensor(args, "residual", (c.M, c.N), self.dtype, (c.ldr, 1))
        self._tensor(args, "Y", (c.M, c.N), self.dtype, (c.ldy, 1))
        self._workspace(args)

    def run(self, args: Args, stream: Optional[int] = None) -> None:
        self._call("run", args, stream)

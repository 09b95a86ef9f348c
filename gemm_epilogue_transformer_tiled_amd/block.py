"""Binding of libge_block.so: the transformer-block operators around the fused products.

The gated feed-forward block with its backward pass (``GatedFFN``).  The functions carry the C
names of ``include/ge_block.h``; the classes own one handle and its zero-filled workspace, like
``Plan``.  Argument marshalling only: every step of the computation runs in the HIP kernels.
The classes check shapes, strides, element types and devices of the tensors they are given; the
library checks pointers and sizes again.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional

import torch

from . import ACT_NAMES, GE_LAYOUT_KN, GE_LAYOUT_NK, GE_OK, GemmEpilogueError

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libge_block.so")

GE_FFN_TILE_256, GE_FFN_TILE_128, GE_FFN_TILE_64, GE_FFN_TILE_COUNT = range(4)
LAYOUT_NAMES = {"kn": GE_LAYOUT_KN, "nk": GE_LAYOUT_NK}

_p, _i32, _i64, _f, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class ge_ffn_desc_t(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("M", "d", "h", "ldx", "ldy", "ldr", "ldg", "lddy", "lddx",
                                    "ldw", "ldwd", "lddw", "lddwd")] + \
               [(n, _i32) for n in ("act", "w_layout", "residual", "save", "tile")]


class ge_ffn_args_t(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("X", "Wg", "Wu", "Wd", "residual", "Y", "G", "U", "dY", "dX", "dWg", "dWu", "dWd",
                                  "workspace")] + [("workspace_bytes", _sz)]


_SIGS = {
    "ge_ffn_validate": ([ctypes.POINTER(ge_ffn_desc_t)], ctypes.c_int),
    "ge_ffn_create": ([ctypes.POINTER(ge_ffn_desc_t), ctypes.POINTER(_p)], ctypes.c_int),
    "ge_ffn_workspace_size": ([_p, _i32, ctypes.POINTER(_sz)], ctypes.c_int),
    "ge_ffn_forward": ([_p, ctypes.POINTER(ge_ffn_args_t), _p], ctypes.c_int),
    "ge_ffn_backward": ([_p, ctypes.POINTER(ge_ffn_args_t), _p], ctypes.c_int),
    "ge_ffn_destroy": ([_p], None),
    "ge_ffn_describe": ([_p, ctypes.c_char_p, _sz], ctypes.c_int),
}
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


def _check(status: int, where: str) -> None:
    if status != GE_OK:
        raise GemmEpilogueError(status, where)


class Args:
    """A pack of device pointers (``.c``, the C struct) and the tensors behind them, which it
    keeps alive.  Build it once and pass it to every call on those tensors."""

    def __init__(self, struct: ctypes.Structure, tensors: Dict[str, Optional[torch.Tensor]]):
        self.c = struct
        self.tensors = tensors
        self._ref = ctypes.byref(struct)
        self._fits = {}          # plan -> the calls whose tensors were found to fit it
        for name, t in tensors.items():
            if hasattr(struct, name):
                setattr(struct, name, None if t is None else t.data_ptr())


class _Plan:
    """What the operators' classes share: the handle, the workspace, the device and the checks."""

    _destroy = None

    def __init__(self, device):
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.handle = None

    def _scratch(self, nbytes: int) -> torch.Tensor:
        """A zero-filled workspace that stays where it is as long as the plan lives (captured graphs
        hold its address)."""
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the plan's workspace is made by its first call: call it once before the capture, "
                               "or give the arguments a workspace")
        return torch.zeros(nbytes, dtype=torch.uint8, device=self.device)

    def _stream(self, stream: Optional[int]) -> int:
        return torch.cuda.current_stream(self.device).cuda_stream if stream is None else stream

    def _tensor(self, args: Args, name: str, shape, dtype, strides=None, optional=False) -> None:
        """Raises ValueError unless tensor `name` is on the plan's device with this shape and type,
        and these strides (default: any; the stride of an extent below two does not matter)."""
        t = args.tensors.get(name)
        if t is None:
            if optional or 0 in shape:
                return
            raise ValueError(f"{name} is missing")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the plan on {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} is {t.dtype}, not {dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        for n, have, want in zip(shape, t.stride(), strides or ()) if t.numel() else ():
            if n > 1 and want is not None and have != want:
                raise ValueError(f"{name} has strides {t.stride()}, the plan {tuple(strides)}")

    def close(self) -> None:
        if self.handle:
            getattr(lib, self._destroy)(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def make_ffn_args(X=None, Wg=None, Wu=None, Wd=None, residual=None, Y=None, G=None, U=None, dY=None, dX=None,
                  dWg=None, dWu=None, dWd=None, workspace=None) -> Args:
    """Pointer pack of the feed-forward block from bf16 device tensors (None: not used)."""
    a = Args(ge_ffn_args_t(), dict(X=X, Wg=Wg, Wu=Wu, Wd=Wd, residual=residual, Y=Y, G=G, U=U, dY=dY, dX=dX,
                                   dWg=dWg, dWu=dWu, dWd=dWd, workspace=workspace))
    a.c.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return a


def make_ffn_desc(M: int, d: int, h: int, act: str = "silu", w_layout: str = "kn", residual: bool = False,
                  save: bool = False, tile: Optional[int] = None, **ld: int) -> ge_ffn_desc_t:
    """Descriptor for packed row-major tensors; ``ld``: leading dimensions that differ (ldx, ldy, ldr,
    ldg, lddy, lddx, ldw, ldwd, lddw, lddwd).  tile: a ge_ffn_tile_t (None: chosen by size)."""
    desc = ge_ffn_desc_t(M=M, d=d, h=h, act=ACT_NAMES[act], w_layout=LAYOUT_NAMES[w_layout], residual=int(residual),
                         save=int(save), tile=0 if tile is None else tile + 1)
    wi, wo = (h, d) if w_layout == "kn" else (d, h)
    base = dict(ldx=d, ldy=d, ldr=d, ldg=h, lddy=d, lddx=d, ldw=wi, ldwd=wo, lddw=wi, lddwd=wo)
    for name in ld:
        if name not in base:
            raise TypeError(f"unknown leading dimension {name}")
    for name, value in {**base, **ld}.items():
        setattr(desc, name, value)
    return desc


class GatedFFN(_Plan):
    """The gated feed-forward block Y = (act(X Wg) * (X Wu)) Wd (+ R) for M rows, and its gradients.

    ``forward`` reads X, Wg, Wu, Wd (and ``residual``), writes Y and, with ``save``, G and U;
    ``backward`` reads X, Wg, Wu, Wd, G, U, dY and writes dX, dWg, dWu, dWd (dX None: not computed;
    the three weight gradients None: not computed).  Calls run on the current stream unless one is
    given; those that share this plan's workspace must be ordered (give concurrent calls, and
    graphs that replay at once, arguments with workspaces of their own)."""

    _destroy = "ge_ffn_destroy"

    def __init__(self, M: int, d: int, h: int, act: str = "silu", w_layout: str = "kn", residual: bool = False,
                 save: bool = False, tile: Optional[int] = None, device="cuda", **ld: int):
        super().__init__(device)
        self.desc = make_ffn_desc(M, d, h, act, w_layout, residual, save, tile, **ld)
        out = _p()
        _check(lib.ge_ffn_create(ctypes.byref(self.desc), ctypes.byref(out)), "ge_ffn_create")
        self.handle = out.value
        # forward and backward share one workspace in a training plan; a plan without `save` whose
        # backward is called gets a second one
        self.workspace = self._scratch(max(self.workspace_size(b) for b in ((False, True) if save else (False,))))
        self.workspace_backward = self.workspace if save else None

    def workspace_size(self, backward: bool = False) -> int:
        n = _sz()
        _check(lib.ge_ffn_workspace_size(self.handle, int(backward), ctypes.byref(n)), "ge_ffn_workspace_size")
        return n.value

    def describe(self) -> str:
        buf = ctypes.create_string_buffer(256)
        _check(lib.ge_ffn_describe(self.handle, buf, len(buf)), "ge_ffn_describe")
        return buf.value.decode()

    def _fit(self, args: Args, backward: bool) -> None:
        c, bf16 = self.desc, torch.bfloat16
        M, d, h = c.M, c.d, c.h
        kn = c.w_layout == GE_LAYOUT_KN
        wi, wo = ((d, h), (h, d)) if kn else ((h, d), (d, h))
        dw = backward and any(args.tensors.get(n) is not None for n in ("dWg", "dWu", "dWd"))
        dx = backward and args.tensors.get("dX") is not None
        if not backward or dw:
            self._tensor(args, "X", (M, d), bf16, (c.ldx, 1))
        if not backward or dx:
            self._tensor(args, "Wg", wi, bf16, (c.ldw, 1))
            self._tensor(args, "Wu", wi, bf16, (c.ldw, 1))
        self._tensor(args, "Wd", wo, bf16, (c.ldwd, 1))
        if backward or c.save:
            self._tensor(args, "G", (M, h), bf16, (c.ldg, 1))
            self._tensor(args, "U", (M, h), bf16, (c.ldg, 1))
        if backward:
            self._tensor(args, "dY", (M, d), bf16, (c.lddy, 1))
            self._tensor(args, "dX", (M, d), bf16, (c.lddx, 1), optional=True)
            if dw:
                self._tensor(args, "dWg", wi, bf16, (c.lddw, 1))
                self._tensor(args, "dWu", wi, bf16, (c.lddw, 1))
                self._tensor(args, "dWd", wo, bf16, (c.lddwd, 1))
        else:
            self._tensor(args, "Y", (M, d), bf16, (c.ldy, 1))
            if c.residual:
                self._tensor(args, "residual", (M, d), bf16, (c.ldr, 1))
        if backward and args.tensors["workspace"] is None and self.workspace_backward is None:
            self.workspace_backward = self._scratch(self.workspace_size(True))

    def _run(self, args: Args, backward: bool, stream: Optional[int]) -> None:
        fits = args._fits.get(self, ())
        if backward not in fits:
            self._fit(args, backward)
            args._fits[self] = (*fits, backward)
        if args.tensors["workspace"] is None:
            ws = self.workspace_backward if backward else self.workspace
            args.c.workspace, args.c.workspace_bytes = ws.data_ptr(), ws.numel()
        call = lib.ge_ffn_backward if backward else lib.ge_ffn_forward
        st = call(self.handle, args._ref, self._stream(stream))
        if st != GE_OK:
            raise GemmEpilogueError(st, "ge_ffn_backward" if backward else "ge_ffn_forward")

    def forward(self, args: Args, stream: Optional[int] = None) -> None:
        self._run(args, False, stream)

    def backward(self, args: Args, stream: Optional[int] = None) -> None:
        self._run(args, True, stream)

"""Binding of libge_block.so: the transformer-block operators around the fused products.

The gated feed-forward block with its backward pass (``GatedFFN``), the per-head norm of queries and
keys with the position rotation and its gradient (``QKRotary``), the global gradient norm with
clipping (``GradClip``).  ``lib`` holds the C functions of ``include/ge_block.h``; the classes own one handle and its zero-filled workspace, like
``Plan``.  A call may run on any stream of the plan's device; as with tensors used on a stream that is not their own, a plan is kept
until its calls on other streams than the current one have run, and as long as a graph that holds them.
Argument marshalling only: every step of the computation runs in the HIP kernels.
The classes check shapes, strides, element types and devices of the tensors they are given; the
library checks pointers and sizes again.
"""
from __future__ import annotations

import ctypes
import os
import math
from typing import Dict, Optional, Sequence, Tuple

import torch

from . import ACT_NAMES, GE_DT_BF16, GE_DT_FP32, GE_LAYOUT_KN, GE_LAYOUT_NK, GE_OK, GemmEpilogueError

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libge_block.so")

GE_FFN_TILE_256, GE_FFN_TILE_128, GE_FFN_TILE_64, GE_FFN_TILE_COUNT = range(4)
GE_PAIRS_INTERLEAVED, GE_PAIRS_HALF = range(2)
PAIR_NAMES = {"interleaved": GE_PAIRS_INTERLEAVED, "half": GE_PAIRS_HALF}
DTYPES = {torch.bfloat16: GE_DT_BF16, torch.float32: GE_DT_FP32}
LAYOUT_NAMES = {"kn": GE_LAYOUT_KN, "nk": GE_LAYOUT_NK}

_p, _i32, _i64, _f, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class ge_ffn_desc_t(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("M", "d", "h", "ldx", "ldy", "ldr", "ldg", "lddy", "lddx",
                                    "ldw", "ldwd", "lddw", "lddwd")] + \
               [(n, _i32) for n in ("act", "w_layout", "residual", "save", "tile")]


class ge_ffn_args_t(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("X", "Wg", "Wu", "Wd", "residual", "Y", "G", "U", "dY", "dX", "dWg", "dWu", "dWd",
                                  "workspace")] + [("workspace_bytes", _sz)]


class ge_qk_desc_t(ctypes.Structure):
    _fields_ = [(n, _i64) for n in ("tokens", "heads_q", "heads_k", "q_token", "q_head", "k_token", "k_head",
                                    "oq_token", "oq_head", "ok_token", "ok_head",
                                    "dq_token", "dq_head", "dk_token", "dk_head")] + \
               [(n, _i32) for n in ("head_dim", "rot_dim", "pairs", "norm", "dtype", "pos64")] + [("eps", _f)]


class ge_qk_args_t(ctypes.Structure):
    _fields_ = [(n, _p) for n in ("q", "k", "q_out", "k_out", "positions", "inv_freq", "gain_q", "gain_k",
                                  "dq_out", "dk_out", "dq", "dk", "dgain_q", "dgain_k", "workspace")] + \
               [("workspace_bytes", _sz), ("amplitude", _f)]


class ge_clip_tensor_t(ctypes.Structure):
    _fields_ = [("numel", _i64), ("dtype", _i32)]


class ge_clip_args_t(ctypes.Structure):
    _fields_ = [("in_", _p), ("out", _p), ("norm", _p), ("workspace", _p), ("workspace_bytes", _sz),
                ("max_norm", _f), ("eps", _f)]


_SIGS = {
    "ge_ffn_validate": ([ctypes.POINTER(ge_ffn_desc_t)], ctypes.c_int),
    "ge_ffn_create": ([ctypes.POINTER(ge_ffn_desc_t), ctypes.POINTER(_p)], ctypes.c_int),
    "ge_ffn_workspace_size": ([_p, _i32, ctypes.POINTER(_sz)], ctypes.c_int),
    "ge_ffn_forward": ([_p, ctypes.POINTER(ge_ffn_args_t), _p], ctypes.c_int),
    "ge_ffn_backward": ([_p, ctypes.POINTER(ge_ffn_args_t), _p], ctypes.c_int),
    "ge_ffn_destroy": ([_p], None),
    "ge_ffn_describe": ([_p, ctypes.c_char_p, _sz], ctypes.c_int),
    "ge_qk_validate": ([ctypes.POINTER(ge_qk_desc_t)], ctypes.c_int),
    "ge_qk_create": ([ctypes.POINTER(ge_qk_desc_t), ctypes.POINTER(_p)], ctypes.c_int),
    "ge_qk_workspace_size": ([_p, ctypes.POINTER(_sz)], ctypes.c_int),
    "ge_qk_forward": ([_p, ctypes.POINTER(ge_qk_args_t), _p], ctypes.c_int),
    "ge_qk_backward": ([_p, ctypes.POINTER(ge_qk_args_t), _p], ctypes.c_int),
    "ge_qk_destroy": ([_p], None),
    "ge_clip_create": ([ctypes.POINTER(ge_clip_tensor_t), _i32, ctypes.POINTER(_p)], ctypes.c_int),
    "ge_clip_workspace_size": ([_p, ctypes.POINTER(_sz)], ctypes.c_int),
    "ge_clip_run": ([_p, ctypes.POINTER(ge_clip_args_t), _p], ctypes.c_int),
    "ge_clip_destroy": ([_p], None),
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
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _check(status: int, where: str) -> None:
    if status != GE_OK:
        raise GemmEpilogueError(status, where)


class Args:
    """A pack of device pointers (``.c``, the C struct) and the tensors behind them, which it
    keeps alive, with the plans it was used with and their workspaces.  Build it once and pass it to every
    call on those tensors."""

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

    def _create(self, call, where: str) -> None:
        """Makes the handle with the plan's device current: it belongs to that device."""
        out = _p()
        with torch.cuda.device(self.device):
            _check(call(ctypes.byref(out)), where)
        self.handle = out.value

    def _scratch(self, nbytes: int, stream: Optional[int] = None) -> torch.Tensor:
        """A zero-filled workspace that stays where it is as long as the plan lives (captured graphs
        hold its address).  Taken and cleared on ``stream`` (a handle) where a call needs it, so that the
        call finds it clear; without one on the device's current stream, and waited for: later
        calls may run on any."""
        if stream is None:
            where = torch.cuda.device(self.device)
        else:                                   # (an ExternalStream of handle 0 would be a stream of torch's pool)
            where = torch.cuda.stream(torch.cuda.ExternalStream(stream, device=self.device) if stream
                                      else torch.cuda.default_stream(self.device))
        with where:
            if torch.cuda.is_current_stream_capturing():
                raise RuntimeError("the plan's workspace is made by its first call: call it once before the capture, "
                                   "or give the arguments a workspace")
            workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
            if stream is None:
                torch.cuda.current_stream(self.device).synchronize()
        return workspace

    def _stream(self, stream: Optional[int]) -> int:
        if stream is not None:
            return stream
        if _raw_stream is not None:             # the same handle, without building a Stream object (2 us)
            return _raw_stream(self.device.index)
        return torch.cuda.current_stream(self.device).cuda_stream

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

    def _workspace(self, args: Args) -> None:
        """Raises ValueError unless the pack's workspace, if it has one, is dense memory of the plan's device
        (its size and alignment are the library's to check)."""
        w = args.tensors["workspace"]
        if w is None:
            return
        if w.device != self.device:
            raise ValueError(f"workspace is on {w.device}, the plan on {self.device}")
        if not w.is_contiguous():
            raise ValueError("workspace is not contiguous")

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
        self._create(lambda out: lib.ge_ffn_create(ctypes.byref(self.desc), out), "ge_ffn_create")
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

    def _fit(self, args: Args, backward: bool, stream: int) -> None:
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
        self._workspace(args)
        if backward and args.tensors["workspace"] is None and self.workspace_backward is None:
            self.workspace_backward = self._scratch(self.workspace_size(True), stream)

    def _run(self, args: Args, backward: bool, stream: Optional[int]) -> None:
        stream = self._stream(stream)
        fits = args._fits.get(self, ())
        if backward not in fits:
            self._fit(args, backward, stream)
            args._fits[self] = (*fits, backward)
        if args.tensors["workspace"] is None:
            ws = self.workspace_backward if backward else self.workspace
            args.c.workspace, args.c.workspace_bytes = ws.data_ptr(), ws.numel()
        call = lib.ge_ffn_backward if backward else lib.ge_ffn_forward
        st = call(self.handle, args._ref, stream)
        if st != GE_OK:
            raise GemmEpilogueError(st, "ge_ffn_backward" if backward else "ge_ffn_forward")

    def forward(self, args: Args, stream: Optional[int] = None) -> None:
        self._run(args, False, stream)

    def backward(self, args: Args, stream: Optional[int] = None) -> None:
        self._run(args, True, stream)


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_length: int = 4096, slow: float = 1.0, fast: float = 32.0
                       ) -> Tuple[torch.Tensor, float]:
    """(inv_freq, amplitude) of the rotation: inv_freq[i] = base^(-2i / rot_dim), fp32 on the host, scaled
    for contexts ``factor`` times longer than the original.

    none: as they are.  linear: all divided by factor.  base: base * factor^(rot_dim / (rot_dim - 2)), which
    divides the slowest by factor and leaves the fastest.  by_parts: those that make fewer than ``slow``
    turns over original_length are divided by factor, those that make more than ``fast`` are kept, those
    between are blended, and amplitude is 0.1 ln(factor) + 1 (1 for the others)."""
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim is even and not negative")
    if not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("factor is at least 1")
    if not (base > 0.0 and math.isfinite(base)):
        raise ValueError("base is above 0 and finite")
    if scaling == "by_parts" and not (slow <= fast and original_length > 0):
        raise ValueError("slow is at most fast, original_length above 0")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2)) if rot_dim > 2 else base
    f = base ** (-2.0 * i / max(rot_dim, 1))
    amplitude = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0) if slow < fast else (turns >= slow).double()
        f = f * keep + f / factor * (1.0 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling}")
    return f.float(), amplitude


def make_qk_args(q=None, k=None, q_out=None, k_out=None, positions=None, inv_freq=None, amplitude: float = 1.0,
                 gain_q=None, gain_k=None, dq_out=None, dk_out=None, dq=None, dk=None, dgain_q=None, dgain_k=None,
                 workspace=None) -> Args:
    """Pointer pack of the query/key norm with rotation: tensors [tokens][heads][head_dim] (any strides
    over tokens and heads), gains [head_dim], positions [tokens], inv_freq [rot_dim / 2]."""
    a = Args(ge_qk_args_t(), dict(q=q, k=k, q_out=q_out, k_out=k_out, positions=positions, inv_freq=inv_freq,
                                  gain_q=gain_q, gain_k=gain_k, dq_out=dq_out, dk_out=dk_out, dq=dq, dk=dk,
                                  dgain_q=dgain_q, dgain_k=dgain_k, workspace=workspace))
    a.c.amplitude = amplitude
    a.c.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return a


def _apart(tokens: int, heads: int, head_dim: int, strides: Sequence[int]) -> bool:
    """Whether (token, head) strides keep the heads of all tokens apart, as outputs' strides have to."""
    rows = [(s, n) for s, n in zip(strides, (tokens, heads)) if n != 1]
    if 0 in (tokens, heads) or not rows:
        return True
    (low, n), (high, _) = min(rows), max(rows)
    return low >= head_dim and (len(rows) < 2 or high >= (n - 1) * low + head_dim)


class QKRotary(_Plan):
    """Per-head RMS norm of queries and keys with the position rotation, and its gradient.

    ``forward`` reads q, k, positions, inv_freq (and the gains), writes q_out, k_out (which may be q and
    k); ``backward`` reads dq_out, dk_out (and, with the norm, q, k and the gains), writes dq, dk and, with
    the norm, dgain_q, dgain_k.  ``*_strides``: (token, head) strides in elements, default packed; the
    gradients of the outputs have the outputs' strides, dq and dk those of q and k unless given, or packed
    where q and k repeat elements (an expanded tensor)."""

    _destroy = "ge_qk_destroy"

    def __init__(self, tokens: int, heads_q: int, heads_k: int, head_dim: int, rot_dim: Optional[int] = None,
                 pairs: str = "half", norm: bool = True, eps: float = 1e-6, dtype=torch.bfloat16,
                 q_strides: Optional[Sequence[int]] = None, k_strides: Optional[Sequence[int]] = None,
                 q_out_strides: Optional[Sequence[int]] = None, k_out_strides: Optional[Sequence[int]] = None,
                 dq_strides: Optional[Sequence[int]] = None, dk_strides: Optional[Sequence[int]] = None,
                 positions_dtype=torch.int64, device="cuda"):
        super().__init__(device)
        if dtype not in DTYPES:
            raise ValueError(f"element type {dtype}: bfloat16 or float32")
        if positions_dtype not in (torch.int32, torch.int64):
            raise ValueError(f"positions of type {positions_dtype}: int32 or int64")
        self.dtype, self.positions_dtype = dtype, positions_dtype
        q = tuple(q_strides or (heads_q * head_dim, head_dim))
        k = tuple(k_strides or (heads_k * head_dim, head_dim))
        oq = tuple(q_out_strides or (heads_q * head_dim, head_dim))
        ok = tuple(k_out_strides or (heads_k * head_dim, head_dim))
        own = lambda s, heads: s if _apart(tokens, heads, head_dim, s) else (heads * head_dim, head_dim)  # noqa: E731
        dq, dk = tuple(dq_strides or own(q, heads_q)), tuple(dk_strides or own(k, heads_k))
        self.strides = dict(q=q, k=k, q_out=oq, k_out=ok, dq_out=oq, dk_out=ok, dq=dq, dk=dk)
        self.desc = ge_qk_desc_t(tokens, heads_q, heads_k, *q, *k, *oq, *ok, *dq, *dk, head_dim,
                                 head_dim if rot_dim is None else rot_dim, PAIR_NAMES[pairs], int(norm), DTYPES[dtype],
                                 int(positions_dtype == torch.int64), eps)
        self._create(lambda out: lib.ge_qk_create(ctypes.byref(self.desc), out), "ge_qk_create")
        n = _sz()
        _check(lib.ge_qk_workspace_size(self.handle, ctypes.byref(n)), "ge_qk_workspace_size")
        self.workspace_bytes = n.value
        self.workspace = None        # made by the first backward

    def _fit(self, args: Args, backward: bool, stream: int) -> None:
        c = self.desc
        T, D = c.tokens, c.head_dim
        names = (("q", "k") if c.norm else ()) + ("dq_out", "dk_out", "dq", "dk") if backward else ("q", "k", "q_out", "k_out")
        for n in names:
            heads = c.heads_q if "q" in n else c.heads_k
            self._tensor(args, n, (T, heads, D), self.dtype, (*self.strides[n], 1))
        if c.rot_dim and T:
            self._tensor(args, "positions", (T,), self.positions_dtype, (1,))
            self._tensor(args, "inv_freq", (c.rot_dim // 2,), torch.float32, (1,))
        if c.norm:
            for s, heads in (("q", c.heads_q), ("k", c.heads_k)):
                if heads:
                    self._tensor(args, "gain_" + s, (D,), self.dtype, (1,))
                if backward:                    # (written without heads too, where it is given)
                    self._tensor(args, "dgain_" + s, (D,), torch.float32, (1,), optional=not heads)
            if backward:
                self._workspace(args)
            if backward and args.tensors["workspace"] is None and self.workspace is None:
                self.workspace = self._scratch(self.workspace_bytes, stream)

    def _run(self, args: Args, backward: bool, stream: Optional[int]) -> None:
        stream = self._stream(stream)
        fits = args._fits.get(self, ())
        if backward not in fits:
            self._fit(args, backward, stream)
            args._fits[self] = (*fits, backward)
        if backward and self.workspace is not None and args.tensors["workspace"] is None:
            args.c.workspace, args.c.workspace_bytes = self.workspace.data_ptr(), self.workspace.numel()
        call = lib.ge_qk_backward if backward else lib.ge_qk_forward
        st = call(self.handle, args._ref, stream)
        if st != GE_OK:
            raise GemmEpilogueError(st, "ge_qk_backward" if backward else "ge_qk_forward")

    def forward(self, args: Args, stream: Optional[int] = None) -> None:
        self._run(args, False, stream)

    def backward(self, args: Args, stream: Optional[int] = None) -> None:
        self._run(args, True, stream)


def make_clip_args(grads: Sequence[torch.Tensor], outs: Optional[Sequence[torch.Tensor]] = None, norm=None,
                   max_norm: float = 1.0, eps: float = 1e-6, workspace=None) -> Args:
    """Pointer pack of the clipping: the gradients, the tensors their clipped values go to (the gradients
    themselves to clip in place; None: only the norm) and a float32 tensor of one element for the norm."""
    grads = list(grads)
    outs = None if outs is None else list(outs)
    if outs is not None and len(outs) != len(grads):
        raise ValueError("as many outputs as gradients")
    a = Args(ge_clip_args_t(), dict(norm=norm, workspace=workspace))
    a.grads, a.outs = grads, outs
    a._in = (_p * max(len(grads), 1))(*[g.data_ptr() for g in grads])
    a.c.in_ = ctypes.cast(a._in, _p)
    if outs is not None:
        a._out = (_p * max(len(outs), 1))(*[g.data_ptr() for g in outs])
        a.c.out = ctypes.cast(a._out, _p)
    a.c.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    a.c.max_norm, a.c.eps = max_norm, eps
    return a


class GradClip(_Plan):
    """The global norm of a list of gradients (bf16 and fp32 mixed, each dense) and their clipping:
    every gradient times min(1, max_norm / (norm + eps)).  Made for a list of tensors of given sizes and
    types; ``run`` takes any pack of tensors like them."""

    _destroy = "ge_clip_destroy"

    def __init__(self, grads: Sequence[torch.Tensor], device=None):
        grads = list(grads)
        super().__init__(device if device is not None else grads[0].device if grads else "cuda")
        for g in grads:
            if g.dtype not in DTYPES:
                raise ValueError(f"gradient of type {g.dtype}: bfloat16 or float32")
        self.like = [(g.numel(), g.dtype) for g in grads]
        table = (ge_clip_tensor_t * max(len(grads), 1))(*[(n, DTYPES[t]) for n, t in self.like])
        self._create(lambda out: lib.ge_clip_create(table, len(grads), out), "ge_clip_create")
        n = _sz()
        _check(lib.ge_clip_workspace_size(self.handle, ctypes.byref(n)), "ge_clip_workspace_size")
        self.workspace = self._scratch(n.value)

    def _fit(self, args: Args) -> None:
        if args.outs is None and args.tensors["norm"] is None:
            raise ValueError("neither a norm nor outputs to write")
        self._workspace(args)
        if args.tensors["norm"] is not None:
            self._tensor(args, "norm", (1,), torch.float32)
        for kind in (args.grads, args.outs):
            if kind is None:
                continue
            if len(kind) != len(self.like):
                raise ValueError(f"{len(kind)} tensors, the plan has {len(self.like)}")
            for i, (g, like) in enumerate(zip(kind, self.like)):
                if (g.numel(), g.dtype) != like:
                    raise ValueError(f"tensor {i} has {g.numel()} values of {g.dtype}, the plan {like}")
                if g.device != self.device:
                    raise ValueError(f"tensor {i} is on {g.device}, the plan on {self.device}")
                if not g.is_contiguous():
                    raise ValueError(f"tensor {i} is not contiguous")

    def run(self, args: Args, stream: Optional[int] = None) -> None:
        if self not in args._fits:
            self._fit(args)
            args._fits[self] = True
        if args.tensors["workspace"] is None:
            args.c.workspace, args.c.workspace_bytes = self.workspace.data_ptr(), self.workspace.numel()
        st = lib.ge_clip_run(self.handle, args._ref, self._stream(stream))
        if st != GE_OK:
            raise GemmEpilogueError(st, "ge_clip_run")

"""libge_rows.so on the host: it loads, exports every symbol its header declares, and its HIP-free
validation accepts and refuses as documented.  No compute is launched here."""
from __future__ import annotations

import ctypes
import math
import os
import re

import pytest
import torch

import gemm_epilogue_transformer_tiled_amd as ge
from gemm_epilogue_transformer_tiled_amd import rows

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = ge.GE_OK, ge.GE_ERR_INVALID_ARG, ge.GE_ERR_UNSUPPORTED


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ge_rows.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(ge_\w+)\s*\(", text)))
    lib = ctypes.CDLL(rows.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert set(names) == set(rows.EXPORTED)


def test_structures_have_the_headers_fields():
    """Same names in the same order as the header's."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ge_rows.h")).read(), flags=re.S)
    for m in re.finditer(r"typedef struct \{(.*?)\}\s*(ge_\w+_t);", text, flags=re.S):
        fields = [re.sub(r"[*\s]", "", n) for decl in m[1].split(";") if decl.strip()
                  for n in re.sub(r"^\s*(const\s+)?\w+(?=[\s*])", "", decl.strip(), count=1).split(",")]
        assert fields == [f[0] for f in getattr(rows, m[2])._fields_], m[2]


def _norm(**kw):
    base = dict(rows=10, d=64, dtype=ge.GE_DT_BF16, residual=1, site=0, dropout=0.1, eps=1e-5)
    base.update(kw)
    for n in ("ldx", "ldr", "lds", "ldy", "lddy", "ldds", "lddx", "lddr"):
        base.setdefault(n, max(base["d"], 0))
    return rows.lib.ge_norm_validate(ctypes.byref(rows.ge_norm_desc_t(**base)))


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(rows=0), OK), (dict(d=1), OK), (dict(d=32768), OK), (dict(d=77, ldx=78), OK), (dict(eps=0.0), OK),
    (dict(dropout=65535 / 65536), OK), (dict(dtype=ge.GE_DT_FP32), OK),
    (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(d=-8), INVALID), (dict(ldx=63), INVALID), (dict(lddr=63), INVALID),
    (dict(residual=2), INVALID), (dict(dtype=7), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(dropout=-0.1), INVALID), (dict(dropout=1.0), INVALID), (dict(dropout=math.nan), INVALID),
    (dict(dtype=ge.GE_DT_FP8_E4M3), UNSUPPORTED), (dict(d=32769), UNSUPPORTED), (dict(rows=1 << 41), UNSUPPORTED),
    (dict(rows=1 << 29), OK), (dict(rows=(1 << 29) + 1), UNSUPPORTED), (dict(rows=(1 << 29) + 1, dropout=0.0), OK),
    (dict(ldx=1 << 41), UNSUPPORTED), (dict(rows=1 << 30, lds=1 << 40, dropout=0.0), UNSUPPORTED),
])
def test_norm_descriptors(kw, want):
    assert _norm(**kw) == want


def _dropout(**kw):
    base = dict(rows=10, d=64, dtype=ge.GE_DT_BF16, residual=0, site=0, p=0.1)
    base.update(kw)
    for n in ("ldx", "ldr", "ldy", "lddy", "lddx"):
        base.setdefault(n, max(base["d"], 0))
    return rows.lib.ge_dropout_validate(ctypes.byref(rows.ge_dropout_desc_t(**base)))


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(rows=0), OK), (dict(d=0), OK), (dict(d=100000, ldx=100001), OK), (dict(p=0.0), OK),
    (dict(rows=-1), INVALID), (dict(d=-1), INVALID), (dict(ldy=63), INVALID), (dict(p=1.0), INVALID), (dict(p=math.nan), INVALID),
    (dict(p=-1e-9), INVALID), (dict(residual=-1), INVALID), (dict(dtype=3), INVALID),
    (dict(dtype=ge.GE_DT_FP8_E4M3), UNSUPPORTED), (dict(rows=1 << 32, d=8), OK), (dict(rows=(1 << 32) + 1, d=8), UNSUPPORTED),
    (dict(rows=1, d=1 << 31), UNSUPPORTED),
])
def test_dropout_descriptors(kw, want):
    assert _dropout(**kw) == want


def _quant(**kw):
    base = dict(rows=10, d=64, dtype=ge.GE_DT_BF16)
    base.update(kw)
    for n in ("ldx", "ldq"):
        base.setdefault(n, max(base["d"], 0))
    return rows.lib.ge_quant_validate(ctypes.byref(rows.ge_quant_desc_t(**base)))


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(rows=0), OK), (dict(d=0), OK), (dict(d=32768), OK), (dict(ldq=65), OK),
    (dict(rows=-1), INVALID), (dict(d=-1), INVALID), (dict(ldx=63), INVALID), (dict(ldq=63), INVALID), (dict(dtype=-1), INVALID),
    (dict(dtype=ge.GE_DT_FP8_E4M3), UNSUPPORTED), (dict(d=32769), UNSUPPORTED), (dict(rows=1 << 41), UNSUPPORTED),
])
def test_quant_descriptors(kw, want):
    assert _quant(**kw) == want


def _i8(**kw):
    base = dict(M=10, N=64, K=128, act=0, bias=0, residual=0, dtype=ge.GE_DT_BF16, tile=0)
    base.update(kw)
    for n, size in (("ldx", "K"), ("ldw", "K"), ("ldy", "N"), ("ldr", "N")):
        base.setdefault(n, max(base[size], 0))
    return rows.lib.ge_i8_validate(ctypes.byref(rows.ge_i8_desc_t(**base)))


@pytest.mark.parametrize("kw,want", [
    (dict(), OK), (dict(M=0), OK), (dict(N=0), OK), (dict(K=0), OK), (dict(K=(1 << 17) - 16), OK), (dict(tile=3), OK),
    (dict(ldx=144, ldw=160, ldy=72, ldr=80), OK), (dict(dtype=ge.GE_DT_FP32), OK),
    (dict(M=-1), INVALID), (dict(N=-8), INVALID), (dict(K=-16), INVALID), (dict(act=4), INVALID), (dict(act=-1), INVALID),
    (dict(bias=2), INVALID), (dict(residual=2), INVALID), (dict(tile=4), INVALID), (dict(tile=-1), INVALID), (dict(dtype=9), INVALID),
    (dict(ldx=112), INVALID), (dict(ldw=112), INVALID), (dict(ldy=56), INVALID), (dict(ldr=56), INVALID),
    (dict(dtype=ge.GE_DT_FP8_E4M3), UNSUPPORTED), (dict(N=60), UNSUPPORTED), (dict(K=120), UNSUPPORTED),
    (dict(K=1 << 17), UNSUPPORTED), (dict(ldx=136), UNSUPPORTED), (dict(ldw=136), UNSUPPORTED), (dict(ldy=68), UNSUPPORTED),
    (dict(ldx=1 << 22), UNSUPPORTED), (dict(ldy=1 << 21), OK), (dict(ldy=1 << 21, dtype=ge.GE_DT_FP32), UNSUPPORTED),
    (dict(M=1 << 31), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED), (dict(M=(1 << 31) - 1024, N=1 << 20), UNSUPPORTED),
    (dict(M=(1 << 31) - 1024, N=8, tile=1 + rows.GE_I8_TILE_64), UNSUPPORTED), (dict(M=(1 << 31) - 1024, N=8), OK),
])
def test_i8_descriptors(kw, want):
    assert _i8(**kw) == want


def test_null_handles_and_arguments():
    lib = rows.lib
    n = ctypes.c_size_t()
    for kind in ("norm", "dropout", "quant", "i8"):
        assert getattr(lib, f"ge_{kind}_validate")(None) == INVALID
        assert getattr(lib, f"ge_{kind}_create")(None, None) == INVALID
        out = ctypes.c_void_p(5)
        assert getattr(lib, f"ge_{kind}_create")(None, ctypes.byref(out)) == INVALID and not out.value
        getattr(lib, f"ge_{kind}_destroy")(None)
    assert lib.ge_norm_workspace_size(None, ctypes.byref(n)) == INVALID
    assert lib.ge_i8_workspace_size(None, ctypes.byref(n)) == INVALID
    for f in (lib.ge_norm_forward, lib.ge_norm_backward, lib.ge_dropout_forward, lib.ge_dropout_backward, lib.ge_quant_run,
              lib.ge_i8_run):
        assert f(None, None, None) == INVALID
    assert lib.ge_i8_describe(None, None, 0) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="the refusal without a device")
def test_no_device():
    d = rows.ge_quant_desc_t(rows=1, d=8, ldx=8, ldq=8, dtype=ge.GE_DT_BF16)
    out = ctypes.c_void_p(5)
    assert rows.lib.ge_quant_create(ctypes.byref(d), ctypes.byref(out)) == ge.GE_ERR_DEVICE and not out.value

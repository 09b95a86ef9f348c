"""The largest sizes that include/ge_rows.h names, and the first ones past them."""
from __future__ import annotations

import ctypes

import pytest

import gemm_epilogue_transformer_tiled_amd as ge
from gemm_epilogue_transformer_tiled_amd import rows

OK, UNSUPPORTED = ge.GE_OK, ge.GE_ERR_UNSUPPORTED
PITCHES = {"norm": ("ldx", "ldr", "lds", "ldy", "lddy", "ldds", "lddx", "lddr"), "dropout": ("ldx", "ldr", "ldy", "lddy", "lddx"),
           "quant": ("ldx", "ldq")}


def validate(kind, **kw):
    desc = getattr(rows, f"ge_{kind}_desc_t")
    return getattr(rows.lib, f"ge_{kind}_validate")(ctypes.byref(desc(dtype=ge.GE_DT_BF16, **kw)))


def of_rows(kind, n, d, **kw):
    return validate(kind, rows=n, d=d, **{**dict.fromkeys(PITCHES[kind], d), **kw})


@pytest.mark.parametrize("kind", list(PITCHES))
def test_rows_and_leading_dimensions(kind):
    least = 0 if kind == "dropout" else 1              # (dropout's counters allow no more than 2^32 blocks)
    assert of_rows(kind, 1 << 40, least) == OK
    assert of_rows(kind, (1 << 40) + 1, least) == UNSUPPORTED
    for ld in PITCHES[kind]:
        assert of_rows(kind, 4, 8, **{ld: 1 << 40}) == OK
        assert of_rows(kind, 4, 8, **{ld: (1 << 40) + 1}) == UNSUPPORTED
        assert of_rows(kind, 10 ** 9, 8, **{ld: 10 ** 9}) == OK
        assert of_rows(kind, 10 ** 9 + 1, 8, **{ld: 10 ** 9}) == UNSUPPORTED


def test_columns():
    assert of_rows("dropout", 16, (1 << 31) - 16) == OK
    assert of_rows("dropout", 16, (1 << 31) - 15) == UNSUPPORTED
    assert of_rows("dropout", 16 + 1, (1 << 31) - 16) == UNSUPPORTED      # 2^32 blocks and more
    for kind in ("norm", "quant"):
        assert of_rows(kind, 1, 32768) == OK and of_rows(kind, 1, 32769) == UNSUPPORTED


@pytest.mark.parametrize("tile,rows_of_it,most", [(0, 256, (1 << 23) - 1), (1, 256, (1 << 23) - 1), (2, 128, (1 << 23) - 1),
                                                  (3, 64, (1 << 24) - 1)])
def test_tiles_of_the_int8_product(tile, rows_of_it, most):
    i8 = lambda M, N: validate("i8", M=M, N=N, K=16, ldx=16, ldw=16, ldy=N, ldr=N, tile=tile)  # noqa: E731
    N = 2 * rows_of_it + 8                             # three columns of tiles
    M = most // 3 * rows_of_it
    assert i8(M, N) == OK
    assert i8(M + rows_of_it, N) == UNSUPPORTED
    assert i8((1 << 31) - 513, 8) == (OK if rows_of_it == 256 else UNSUPPORTED)
    assert i8((1 << 31) - 512, 8) == UNSUPPORTED

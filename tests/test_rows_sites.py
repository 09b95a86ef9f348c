"""A dropout's site is 32 bits: what does not fit is refused, not cut to the number of another site."""
from __future__ import annotations

import pytest

from gemm_epilogue_transformer_tiled_amd import rows

MAKE = {"norm": lambda site: rows.LayerNorm(4, 16, dropout=0.1, site=site, device="cpu"),
        "dropout": lambda site: rows.Dropout(4, 16, 0.1, site=site, device="cpu")}


@pytest.mark.parametrize("which", list(MAKE))
def test_sites(which, monkeypatch):
    monkeypatch.setattr(rows._RowsPlan, "_make", lambda self: None)
    for site in (0, 1, 0x7FFFFFFF, 0x80000000, 0xFFFFFFFF):
        assert MAKE[which](site).desc.site == site
    for site in (-1, 1 << 32, (1 << 32) + 1, 1 << 64):
        with pytest.raises(ValueError, match="site"):
            MAKE[which](site)

"""The int8 product over the range of scales that its header names: the row's scale is taken first, and an int32 sum
times any fp32 scale loses nothing to underflow."""
from __future__ import annotations

import pytest
import torch

from tests import rows_parity as rp

pytestmark = pytest.mark.gpu

rows = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.rows")

TILES = [None, rows.GE_I8_TILE_256, rows.GE_I8_TILE_128, rows.GE_I8_TILE_64]


@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("M,K", [(7, 528), (7, 131056), (70, 528)])
def test_scales_far_apart(M, K, tile):
    """x_scale from the least subnormal number to 1e29, w_scale so that the outputs are ordinary: at most four fp32
    roundings of the scaled sum, as for other scales."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N = 264
    gen = torch.Generator("cuda").manual_seed(M + K)
    code = lambda *s: torch.randint(-128, 128, s, generator=gen, device="cuda").to(torch.int8)  # noqa: E731
    X, W = code(M, K), code(N, K)
    X[0], W[0] = -128, -128                            # the largest sum
    for x, w in ((2.0 ** -149, 1e38), (3e-45, 3e30), (1e-38, 1e30), (1e-20, 1e12), (1.0, 1e-4), (1e29, 1e-34), (1e29, 1e-38)):
        xs, ws = torch.full((M,), x, device="cuda"), torch.full((N,), w, device="cuda")
        xs[1::2] *= -1
        Y = torch.empty(M, N, device="cuda")
        plan = rows.Int8Linear(M, N, K, dtype=torch.float32, tile=tile)
        plan.run(rows.make_i8_args(X=X, W=W, x_scale=xs, w_scale=ws, Y=Y))
        ref, tol = rp.int8(X, W, xs, ws, None, None, "none", torch.float32)
        assert bool(ref.ne(0).any()) and bool(Y.isfinite().all())
        rp.check(Y, ref, tol, (x, w))

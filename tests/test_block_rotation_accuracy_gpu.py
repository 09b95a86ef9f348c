"""What the rotation loses to 32 bits, on the GPU: the angles' rounding, and norms of very small heads."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

block = pytest.importorskip("gemm_epilogue_transformer_tiled_amd.block")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def test_angles_are_not_rounded_to_a_fp32_turn():
    """Pairs (1, 0) come out as (cos, sin).  To first order sin * (cos - got) + cos * (got - sin) is the angle
    the kernel turned too far.  A turn t in [-1/2, 1/2] rounded to fp32 is too far by d = 2 pi (fp32(t) - t), up to
    2 pi 2^-26 = 9.4e-8 and on average (over t) more than 2e-8 in size; the sine's own errors do not follow
    d's sign.  Each is below B = 2^-21 (a few units of 2^-24, either function), so over n angles of random sign the
    mean of the excess along d's sign stays within 6 B / sqrt(n), 5e-9 here, unless the rounding is in it."""
    T, D = 5000, 128
    gen = torch.Generator("cuda").manual_seed(11)
    x = torch.zeros(T, 1, D, device="cuda")
    x[..., :D // 2] = 1.0
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, device="cuda")
    inv = block.rotary_frequencies(D)[0].cuda()
    out = torch.empty_like(x)
    block.QKRotary(T, 1, 0, D, norm=False, dtype=torch.float32).forward(
        block.make_qk_args(q=x, q_out=out, positions=pos, inv_freq=inv))
    angle = pos.double()[:, None] * inv.double()[None, :]
    cos, sin, got = angle.cos(), angle.sin(), out[:, 0].double()
    excess = sin * (cos - got[:, :D // 2]) + cos * (got[:, D // 2:] - sin)
    turns = angle / (2 * math.pi)
    turns = turns - turns.round()
    d = 2 * math.pi * (turns.float().double() - turns)
    n = excess.numel()
    assert float(excess.abs().max()) <= 2.0 ** -21
    assert float(d.abs().mean()) > 2e-8
    assert abs(float((excess * d.sign()).mean())) <= 6 * 2.0 ** -21 / math.sqrt(n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("x", [1e-17, 1e-18, 1e-19, 1e-20, 1e-21])
@pytest.mark.parametrize("eps", [0.0, 1e-42])
def test_norm_of_very_small_heads(x, eps, dtype):
    """Without an eps to speak of, heads whose mean square is subnormal are normalised all the same.  Results
    below 2^-126 are multiples of 2^-149, a unit: the D products are each off by half of one, sums of multiples are exact, so
    the mean is off by half a unit from them, half from its own rounding and half from eps's: less than 2, and
    its root by 1 / mean units relative.  Everything else is off by a few 2^-24."""
    D = 64
    q = torch.full((3, 2, D), x, device="cuda", dtype=dtype)
    q[:, :, 1::2] *= -1
    q[1] *= 2
    out, dq = torch.empty_like(q), torch.empty_like(q)
    gain = torch.ones(D, device="cuda", dtype=dtype)
    plan = block.QKRotary(3, 2, 0, D, rot_dim=0, eps=eps, dtype=dtype)
    plan.forward(block.make_qk_args(q=q, q_out=out, gain_q=gain))
    v = q.double()
    mean = v.square().mean(-1, keepdim=True) + eps
    want = v / mean.sqrt()
    unit = 2.0 ** -149
    loss = unit / mean + 16 * 2.0 ** -24 + torch.finfo(dtype).eps / 2
    assert bool(((out.double() - want).abs() <= want.abs() * loss).all()), (float(out[0, 0, 0]), float(want[0, 0, 0]))
    dout = torch.zeros_like(q)
    dout[..., 0] = 1.0
    dgain = torch.empty(D, device="cuda")
    plan.backward(block.make_qk_args(q=q, gain_q=gain, dq_out=dout, dq=dq, dgain_q=dgain))
    n, r = want, 1 / mean.sqrt()
    e = dout.double()
    size = r * (e.abs() + n.abs() * (e * n).abs().mean(-1, keepdim=True))
    assert bool(((dq.double() - r * (e - n * (e * n).mean(-1, keepdim=True))).abs() <= size * (3 * loss)).all())
    assert dgain.isfinite().all()

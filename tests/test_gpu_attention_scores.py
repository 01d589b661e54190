"""Attention with scores far from zero (MI355X only). Queries and keys are
small whole numbers times powers of two, so that every score before the scale
is exact in fp32 and the float64 form has the same; with s the scores and m a
row's largest, a probability's exponent (s - m) scale is rounded twice (2 U of
itself), its exponential and its sums cost a few U more."""
import math

import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import block_reference as R

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _whole(B, Lq, Lk, H, Hk, D, dtype, seed, power=0, most=2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *s: torch.randint(-most, most + 1, s, device="cuda", generator=gen).float()   # noqa: E731
    q, k = draw(B, Lq, H, D) * 2.0 ** power, draw(B, Lk, Hk, D) * 2.0 ** power
    v = torch.randn(B, Lk, Hk, D, device="cuda", generator=gen)
    return q.to(dtype), k.to(dtype), v.to(dtype)


def _exact(q, k, v, mask, causal, scale):
    """{name: (value, error)} of o and lse."""
    B, Lq, H, D = q.shape
    Lk, group, dt = k.shape[1], H // k.shape[2], q.dtype
    half = R.half_step(dt)
    o, e_o = (torch.zeros(B, Lq, H, D, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, e_lse = (torch.zeros(B, H, Lq, dtype=torch.float64, device="cuda") for _ in range(2))
    for b in range(B):
        see = R.visible(Lq, Lk, causal, None if mask is None else mask[b], "cuda")
        for h in range(H):
            k1, v1 = k[b, :, h // group].double(), v[b, :, h // group].double()
            s = torch.where(see, torch.mm(q[b, :, h].double(), k1.t().contiguous()) * scale, -math.inf)
            m = s.amax(1, keepdim=True)
            live = m > -math.inf
            far = torch.where(see, s - m, 0.0)
            p = torch.where(see, torch.exp(far), 0.0)
            total = p.sum(1, keepdim=True).clamp(min=1e-300)
            e_p = p * ((far.abs() + 16) * 4 * R.U + 8 * R.U)
            o[b, :, h] = torch.mm(p, v1) / total
            off = torch.mm(p * (half + (Lk + 8) * R.U) + e_p, v1.abs()) + e_p.sum(1, keepdim=True) * torch.mm(p, v1.abs()) / total
            off = off / total + (2.0 ** -25 * torch.mm(see.double(), v1.abs()) if dt == HF else 0.0)
            e_o[b, :, h] = R.rounded(o[b, :, h], off, dt)
            lse[b, h] = torch.where(live, m + torch.log(total), -math.inf)[:, 0]
            e_lse[b, h] = (e_p.sum(1) / total[:, 0] + (Lk + 8) * R.U) * live[:, 0] + 4 * R.U * lse[b, h].abs().clamp(max=1e37)
    return {"o": (o, e_o), "lse": (lse, e_lse)}


SHAPES = [
    (2, 90, 150, 4, 2, 24, True, True),        # two ways
    (1, 1, 900, 4, 2, 64, False, False),       # keys in parts
    (1, 40, 3000, 2, 2, 128, True, True),
    (1, 200, 300, 2, 2, 64, False, True),
    (1, 1500, 130, 22, 22, 128, False, False), # workgroups of eight waves
    (1, 700, 90, 6, 6, 96, True, False),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scale", [0.3, 2.0 ** 10, 2.0 ** 24 * 1.1, 2.0 ** 28 * 1.3, 2.0 ** 40 * 1.7, 2.0 ** 64])
@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D,causal,masked", SHAPES)
def test_scales(B, Lq, Lk, H, Hk, D, causal, masked, scale, dtype):
    q, k, v = _whole(B, Lq, Lk, H, Hk, D, dtype, D + Lq)
    scale = torch.tensor(scale).item()   # (an fp32 number)
    mask = torch.rand(B, Lk, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) < 0.6 if masked else None
    o, lse = S.attention_forward(q, k, v, key_mask=mask, causal=causal, scale=scale)
    ref = _exact(q, k, v, mask, causal, scale)
    R.check(o, ref["o"], "o")
    R.check(lse, ref["lse"], "lse")


@pytest.mark.parametrize("dtype,power", [(BF, 10), (BF, 14), (BF, 20), (BF, 50), (HF, 10), (HF, 14)])
@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D,causal,masked", SHAPES[:4])
def test_large_queries_and_keys(B, Lq, Lk, H, Hk, D, causal, masked, dtype, power):
    """The same at an ordinary scale, from queries and keys that are large."""
    q, k, v = _whole(B, Lq, Lk, H, Hk, D, dtype, D + Lq, power)
    mask = torch.rand(B, Lk, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) < 0.6 if masked else None
    o, lse = S.attention_forward(q, k, v, key_mask=mask, causal=causal, scale=0.125)
    ref = _exact(q, k, v, mask, causal, 0.125)
    R.check(o, ref["o"], "o")
    R.check(lse, ref["lse"], "lse")


@pytest.mark.parametrize("dtype", [BF, HF])
def test_rows_of_one_tile_far_apart(dtype):
    """Rows with ordinary scores beside rows whose scores are far from zero,
    and keys whose scores rise past that border from tile to tile."""
    q, k, v = _whole(1, 128, 600, 2, 2, 64, dtype, 3)
    q[:, 5::7] *= 2.0 ** 12
    scale = torch.tensor(0.3 * 2.0 ** 12).item()
    q[:, 6::7] *= 2.0 ** -12
    rise = k * torch.exp2(torch.arange(600, device="cuda") // 64).to(dtype)[None, :, None, None]
    for keys in (k, rise, rise.flip(1)):
        o, lse = S.attention_forward(q, keys, v, scale=scale)
        ref = _exact(q, keys, v, None, False, scale)
        R.check(o, ref["o"], "o")
        R.check(lse, ref["lse"], "lse")


@pytest.mark.parametrize("dtype", [BF, HF])
def test_gradients_at_the_largest_scale(dtype):
    q, k, v = _whole(1, 130, 300, 2, 2, 64, dtype, 9, most=1)
    dout = torch.randn(1, 130, 2, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).to(dtype)
    scale = 2.0 ** 10
    o, lse = S.attention_forward(q, k, v, scale=scale)
    ref = R.attention(q, k, v, None, False, scale, (dout, o, lse))
    for name, g in zip(("dq", "dk", "dv"), S.attention_backward(dout, q, k, v, o, lse, scale=scale)):
        R.check(g, ref[name], name)
    with pytest.raises(S.SvdqError):
        S.attention_backward(dout, q, k, v, o, lse, scale=2.0 ** 11)

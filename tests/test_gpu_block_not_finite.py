"""What infinities and NaN do in the calls between a block's linears (MI355X
only): what their formulas say, and no more."""
import math

import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import block_reference as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Lq,Lk,D", [(100, 130, 64), (100, 130, 128), (3, 900, 128), (70, 90, 24)])
def test_attention(Lq, Lk, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(Lk)
    q, k, v = (torch.randn(1, n, 2, D, device="cuda", generator=gen).to(dtype) for n in (Lq, Lk, Lk))
    clean, lse = S.attention_forward(q, k, v)

    def with_value(t, at, value):
        t = t.clone()
        t[at] = value
        return t
    o, l = S.attention_forward(with_value(q, (0, 1, 0, 3), math.nan), k, v)
    assert bool(o[0, 1, 0].isnan().all()) and bool(l[0, 0, 1].isnan())
    rows = torch.arange(Lq, device="cuda") != 1
    assert torch.equal(o[0, rows, 1], clean[0, rows, 1]) and bool(o[0, rows, 0].isfinite().all())
    o, l = S.attention_forward(q, with_value(k, (0, 50, 0, 3), math.nan), v)
    assert bool(o[0, :, 0].isnan().all()) and bool(l[0, 0].isnan().all()) and torch.equal(o[0, :, 1], clean[0, :, 1])
    o, l = S.attention_forward(q, k, with_value(v, (0, 50, 1, 3), math.inf))
    rest = torch.arange(D, device="cuda") != 3
    two = D <= 32 or min(Lq, Lk) <= 64   # probabilities are two values: infinity times a rest below zero
    assert bool((~o[0, :, 1, 3].isfinite() if two else o[0, :, 1, 3] == math.inf).all())
    assert torch.equal(o[..., rest], clean[..., rest]) and torch.equal(l, lse)
    # a key whose score is -infinity has no weight
    q1 = q.clone()
    q1[..., 3] = q1[..., 3].abs() + 0.25
    mask = torch.ones(1, Lk, dtype=torch.bool, device="cuda")
    mask[0, 50] = False
    want = R.attention(q1, k, v, mask, False, D ** -0.5)
    o, l = S.attention_forward(q1, with_value(k, (0, 50, slice(None), 3), -math.inf), v)
    R.check(o, want["o"], "o")
    R.check(l, want["lse"], "lse")


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_residual(value):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, h = (torch.randn(9, 700, device="cuda", generator=gen).to(torch.bfloat16) for _ in range(2))
    rows = torch.arange(9, device="cuda") != 4
    for kind in ("layer", "rms"):
        s, y, _ = S.residual_norm_forward(x, h, kind=kind)
        bad = x.clone()
        bad[4, 600] = value
        s1, y1, _ = S.residual_norm_forward(bad, h, kind=kind)
        assert torch.equal(s1[rows], s[rows]) and torch.equal(y1[rows], y[rows])
        if kind == "rms" and value == math.inf:
            assert bool(y1[4, 600].isnan()) and not bool(y1[4, :600].any()) and not bool(y1[4, 601:].any())
        else:
            assert bool(y1[4].isnan().all())

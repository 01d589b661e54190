"""Launches of more workgroups than a grid's first dimension is given
(MI355X only)."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import fp8_reference as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("more", [0, 1, 5])
def test_row_quantizer_past_a_million_workgroups(more):
    """Every row, the last ones among them, and nothing behind them."""
    M, K = (1 << 22) + more, 16
    g = torch.Generator(device="cuda").manual_seed(more)
    x = torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    q, s = torch.full((M + 9, 128), 7, dtype=torch.uint8, device="cuda"), torch.full((M + 9, 4), 7, dtype=torch.uint8, device="cuda")
    S.fp8_quantize(x[:1])
    S._call("svdq_fp8_quantize", 0, None, x.data_ptr(), M, K, q.data_ptr(), s.data_ptr())
    want, e = R.q8(x.double())
    assert torch.equal(s[:M, 0].double(), e[:, 0] + 127)
    assert torch.equal(q[:M, :K].view(torch.float8_e4m3fn).double(), want * torch.exp2(-e))
    assert bool((q[:M, K:] == 0).all()) and bool((q[M:] == 7).all()) and bool((s[M:] == 7).all())


def test_norm_gradient_of_over_a_million_groups():
    """Groups of one row, the last ones without rows: their gradients are
    zeros, and the gradients of the others their row's alone."""
    M, C, groups = (1 << 20) + 3, 9, (1 << 20) + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = torch.randn(M, C, device="cuda", generator=g), torch.randn(M, C, device="cuda", generator=g)
    mean, rstd = x.mean(1), torch.rand(M, device="cuda", generator=g) + 0.5
    w = torch.rand(groups, C, device="cuda", generator=g)
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=1)
    xhat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    # xhat: a subtraction and a product, then dy xhat: three roundings, and the sums with the other teams' zeros are exact
    want = dy.double() * xhat
    assert bool(((dw[:M].double() - want).abs() <= 3.01 * R.F32 * want.abs()).all())
    assert torch.equal(db[:M], dy) and bool((dw[M:] == 0).all()) and bool((db[M:] == 0).all())
    d = dy.double() * w[:M].double()
    ref = rstd.double()[:, None] * (d - d.mean(1, keepdim=True) - xhat * (d * xhat).mean(1, keepdim=True))
    # the sums of nine values: eight additions, the products' roundings and the division, as in the bound of test_gpu_norm.py
    bound = rstd.double()[:, None] * R.F32 * (6 * d.abs() + 20 * d.abs().mean(1, keepdim=True)
                                              + 26 * xhat.abs() * (d * xhat).abs().mean(1, keepdim=True)) + R.F32 * ref.abs()
    assert bool(((dx.double() - ref).abs() <= bound).all())
    same = S.layer_norm_backward(dy[-50:], x[-50:], mean[-50:], rstd[-50:], w[M - 50:], rows_per_group=1)
    assert torch.equal(same[0], dx[-50:]) and torch.equal(same[1], dw[M - 50:]) and torch.equal(same[2], db[M - 50:])

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

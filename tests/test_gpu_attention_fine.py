"""Attention with probabilities (and ds) as two values at sizes that round them
once otherwise, against float64 (MI355X only); the bounds are derived in
block_reference.py."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import block_reference as R

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D,causal,masked", [
    (1, 130, 300, 4, 2, 64, False, True),
    (2, 300, 260, 4, 1, 128, True, True),
    (1, 1500, 130, 22, 22, 128, False, False),   # whole units
    (13, 300, 300, 20, 20, 64, True, False),
    (22, 150, 290, 12, 6, 96, True, True),
    (1, 700, 700, 2, 2, 72, True, False),
])
def test_against_float64(B, Lq, Lk, H, Hk, D, causal, masked, dtype):
    gen = torch.Generator(device="cuda").manual_seed(Lq + D)
    q, k, v, dout = (torch.randn(B, n, h, D, device="cuda", generator=gen).to(dtype)
                     for n, h in ((Lq, H), (Lk, Hk), (Lk, Hk), (Lq, H)))
    mask = torch.rand(B, Lk, device="cuda", generator=gen) < 0.6 if masked else None
    args = dict(key_mask=mask, causal=causal, fine=True)
    o, lse = S.attention_forward(q, k, v, **args)
    ref = R.attention(q, k, v, mask, causal, D ** -0.5, fine=True)
    R.check(o, ref["o"], "o")
    R.check(lse, ref["lse"], "lse")
    grads = S.attention_backward(dout, q, k, v, o, lse, **args)
    ref = R.attention(q, k, v, mask, causal, D ** -0.5, (dout, o, lse), fine=True)
    for name, g in zip(("dq", "dk", "dv"), grads):
        R.check(g, ref[name], name)
    assert all(torch.equal(a, b) for a, b in zip(grads, S.attention_backward(dout, q, k, v, o, lse, **args)))


def test_workspace_of_the_choice():
    q, k, v, dout = (torch.randn(1, 500, 2, 128, device="cuda").to(BF) for _ in range(4))
    want = S.attention_forward(q, k, v, causal=True, fine=True)
    grads = S.attention_backward(dout, q, k, v, *want, causal=True, fine=True)
    size = (1, 500, 500, 2, 2, 128, BF, True)
    ws = torch.empty(S.attention_workspace_bytes(*size, fine=True), dtype=torch.uint8, device="cuda")
    got = S.attention_forward(q, k, v, causal=True, fine=True, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.empty(S.attention_backward_workspace_bytes(*size, fine=True), dtype=torch.uint8, device="cuda")
    got = S.attention_backward(dout, q, k, v, *want, causal=True, fine=True, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, grads))

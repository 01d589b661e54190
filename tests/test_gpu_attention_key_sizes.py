"""fp16 gradients where keys (or rows) are of very different sizes, against
float64 (MI355X only): a key's ds = p (dout . v - dout . o) follows the largest
values among all keys through o, whatever the key's own values are. The bounds
are derived in block_reference.py; they take the largest |v| of all keys."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import block_reference as R

pytestmark = pytest.mark.gpu

SMALL = [3, 17, 29]   # the keys whose values are small


def _case(B, Lq, Lk, H, Hk, D, ratio, dominant, aligned, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)   # noqa: E731
    q, k, v, dout = rnd(B, Lq, H, D), rnd(B, Lk, Hk, D), rnd(B, Lk, Hk, D), rnd(B, Lq, H, D)
    if aligned:   # dout along the values: dout . o is as large as it can be
        v, dout = v.abs(), dout.abs()
    v[:, SMALL] *= ratio
    if dominant:   # one of them takes most of every row's weight
        q[..., 0] = 4.0
        k[:, SMALL[0], :, 0] += 1.6 * D ** 0.5
    return [t.half() for t in (q, k, v, dout)]


def _check(q, k, v, dout, mask, causal):
    scale = q.shape[3] ** -0.5
    o, lse = S.attention_forward(q, k, v, key_mask=mask, causal=causal)
    grads = S.attention_backward(dout, q, k, v, o, lse, key_mask=mask, causal=causal)
    ref = R.attention(q, k, v, mask, causal, scale, (dout, o, lse))
    for name, g in zip(("dq", "dk", "dv"), grads):
        R.check(g, ref[name], name)


@pytest.mark.parametrize("size", [1.0, 1e-5])
@pytest.mark.parametrize("dominant", [False, True])
@pytest.mark.parametrize("ratio", [1.0, 2.0 ** -6, 2.0 ** -12, 0.0])
@pytest.mark.parametrize("Lq,Lk,H,Hk,D,causal,masked", [
    (130, 200, 4, 2, 24, False, True),      # two operands for ds: heads up to 32
    (130, 200, 2, 2, 64, False, False),     # one operand
    (150, 130, 4, 1, 64, True, True),
    (200, 300, 2, 1, 128, False, True),
    (40, 300, 1, 1, 128, False, False),     # two operands: few rows
    (600, 33, 2, 2, 64, False, True),       # two operands: few keys, the rows in parts
])
def test_keys_of_small_values(Lq, Lk, H, Hk, D, causal, masked, ratio, dominant, size):
    for aligned in (False, True):
        q, k, v, dout = _case(2, Lq, Lk, H, Hk, D, ratio, dominant, aligned, Lq + D)
        mask = None
        if masked:
            mask = torch.rand(2, Lk, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) < 0.7
            mask[:, SMALL] = True
        _check(q, k, v, (dout * size).half(), mask, causal)


@pytest.mark.parametrize("D", [24, 64, 128])
def test_rows_and_keys_of_many_sizes(D):
    """|dout| from 2^-12 to 2^8 over the rows, |v| from 2^-12 to 2^6 over the
    keys, and a masked key whose values are larger than all."""
    q, k, v, dout = _case(1, 200, 260, 4, 2, D, 1.0, False, False, D)
    v = v * torch.exp2(torch.linspace(-12, 6, 260, device="cuda").round())[None, :, None, None].half()
    dout = dout * torch.exp2(torch.linspace(8, -12, 200, device="cuda").round())[None, :, None, None].half()
    mask = torch.ones(1, 260, dtype=torch.bool, device="cuda")
    mask[0, 50] = False
    v[0, 50] = 60000.0
    _check(q, k, v, dout, mask, False)
    _check(q, k, v, dout, mask, True)

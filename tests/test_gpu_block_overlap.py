"""Outputs over inputs of the calls between a block's linears: refused, or the
results of a call with separate outputs (MI355X only)."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S

pytestmark = pytest.mark.gpu


def _rand(*shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(len(shape))).to(torch.bfloat16)


def test_attention():
    q, k, v, dout = _rand(1, 100, 2, 64), _rand(1, 120, 2, 64) * 0.5, _rand(1, 120, 2, 64) * 2, _rand(1, 100, 2, 64) + 1
    for bad in (q, k[:, :100], v[:, 20:]):
        with pytest.raises(ValueError, match="out: overlaps"):
            S.attention_forward(q, k, v, out=bad)
    o, lse = S.attention_forward(q, k, v)
    one = torch.empty_like(k)
    for outs in (dict(dq=q), dict(dq=dout), dict(dq=o), dict(dk=k), dict(dv=v), dict(dk=v), dict(dk=one, dv=one)):
        with pytest.raises(ValueError, match="overlaps"):
            S.attention_backward(dout, q, k, v, o, lse, **outs)
    want = S.attention_backward(dout, q, k, v, o, lse)
    both = torch.empty(1, 120, 4, 64, dtype=torch.bfloat16, device="cuda")   # slices of one buffer lie apart
    got = S.attention_backward(dout, q, k, v, o, lse, dk=both[:, :, ::2], dv=both[:, :, 1::2])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rope_and_residual():
    q, k = _rand(1, 50, 3, 32), _rand(1, 50, 1, 32)
    pos = torch.arange(50, dtype=torch.int32, device="cuda")[:, None]
    freqs = S.rope_frequencies([16])
    want = S.rope(q, k, pos, freqs, [16])
    joint = torch.cat([q, k], 2)
    with pytest.raises(ValueError, match="q_out: overlaps k"):
        S.rope(q, joint[:, :, 3:], pos, freqs, [16], q_out=joint[:, :, 1:])
    with pytest.raises(ValueError, match="is not q itself"):
        S.rope(joint[:, :, :3], None, pos, freqs, [16], q_out=joint[:, :, 1:])
    got = S.rope(joint[:, :, :3], joint[:, :, 3:], pos, freqs, [16], q_out=joint[:, :, :3], k_out=joint[:, :, 3:])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, h = _rand(40, 96), _rand(40, 96) + 1
    with pytest.raises(ValueError, match="s: overlaps x"):
        S.residual_norm_forward(x[:39], h[:39], s=x[1:])
    with pytest.raises(ValueError, match="s: overlaps y"):
        S.residual_norm_forward(x, h, s=x, y=x)
    s, y, stats = S.residual_norm_forward(x, h)
    with pytest.raises(ValueError, match="dx: overlaps dh"):
        S.residual_norm_backward(x, s, h, stats, dx=h, dh=h)
    with pytest.raises(ValueError, match="dh: overlaps h"):
        S.residual_norm_backward(x[1:], s[1:], h[1:], stats[:, 1:].contiguous(), dh=h[:39])

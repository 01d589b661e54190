"""Attention, rotary positions and the gated residual where offsets pass 2^31
and 2^32 elements (MI355X only): against float64, or against a call on the rows
alone."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import block_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free GPU memory")
    yield
    torch.cuda.empty_cache()


def test_attention_over_a_long_cache():
    """Two queries over 2.2 million keys of a cache whose tokens are 2048
    elements apart: 2^32 elements and more."""
    keys, ld, H, HK, D = 2_200_000, 2048, 4, 2, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.zeros(1, keys, ld, dtype=torch.bfloat16, device="cuda")
    kv = cache[:, :, ld - 2 * HK * D:].unflatten(2, (2 * HK, D))
    for at in range(0, keys, 200_000):
        kv[:, at:at + 200_000].normal_(generator=g)
    k, v = kv[:, :, :HK], kv[:, :, HK:]
    k[:, -1] *= 3   # the last keys count
    q = torch.randn(1, 2, H, D, device="cuda", generator=g).to(torch.bfloat16)
    q[:, :, 1] = k[:, -1, :1] * 2
    dout = torch.randn(1, 2, H, D, device="cuda", generator=g).to(torch.bfloat16)
    o, lse = S.attention_forward(q, k, v, causal=True)
    dq, dk, dv = S.attention_backward(dout, q, k, v, o, lse, causal=True)
    ref = R.attention(q, k, v, None, True, D ** -0.5)
    R.check(o, ref["o"], "o")
    R.check(lse, ref["lse"], "lse")
    ref = R.attention(q, k, v, None, True, D ** -0.5, (dout, o, lse))
    for got, name in ((dq, "dq"), (dk, "dk"), (dv, "dv")):
        R.check(got, ref[name], name)
    assert float(lse[0, 1, 1]) > 30   # (the last key's own score)


def test_attention_of_samples_far_apart():
    """Samples 2^32 + 64 elements apart, in the inputs and the outputs."""
    B, L, H, D, ld = 2, 100, 2, 128, (1 << 32) + 64
    g = torch.Generator(device="cuda").manual_seed(2)
    room = [torch.zeros(ld + L * H * D, dtype=torch.float16, device="cuda") for _ in range(3)]
    far = lambda r: torch.as_strided(r, (B, L, H, D), (ld, H * D, D, 1))   # noqa: E731
    q, o = far(room[0]), far(room[1])
    q.normal_(generator=g)
    want, want_lse = S.attention_forward(q.contiguous(), q.contiguous(), q.contiguous())
    got, lse = S.attention_forward(q, q, q, out=o)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    dout = torch.randn(B, L, H, D, device="cuda", generator=g).to(torch.float16)
    want = S.attention_backward(dout, q.contiguous(), q.contiguous(), q.contiguous(), o.contiguous(), lse)
    got = S.attention_backward(dout, q, q, q, o, lse, dq=far(room[2]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rope_of_a_long_stream():
    """300000 tokens of 16384 elements, in place."""
    L, H, D, pairs = 300_000, 128, 128, [64]
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(1, L, H, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    pos = torch.arange(L, device="cuda", dtype=torch.int32)[:, None] * 7
    freqs = S.rope_frequencies(pairs)
    some = [slice(0, 5), slice(131070, 131075), slice(262142, 262147), slice(L - 5, L)]
    want = [R.rope(x[:, r].clone(), pos[r], freqs, pairs, True, False) for r in some]
    S.rope(x, None, pos, freqs, pairs, q_out=x)
    for r, w in zip(some, want):
        R.check(x[:, r], w, "rope")


def test_residual_of_many_wide_rows():
    """300000 x 8192 bf16: a row's results are those of its row alone."""
    M, C = 300_000, 8192
    g = torch.Generator(device="cuda").manual_seed(4)
    x, h = (torch.empty(M, C, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    s, y, stats = S.residual_norm_forward(x, h, kind="rms", post_norm=True)
    dx, dh, *_ = S.residual_norm_backward(y, s, h, stats, kind="rms", post_norm=True, ds=x)
    for r in (slice(0, 7), slice(262140, 262150), slice(M - 7, M)):
        f = [t[r].contiguous() for t in (x, h)]
        s1, y1, st1 = S.residual_norm_forward(*f, kind="rms", post_norm=True)
        dx1, dh1, *_ = S.residual_norm_backward(y1, s1, f[1], st1, kind="rms", post_norm=True, ds=f[0])
        for got, want in ((s, s1), (y, y1), (dx, dx1), (dh, dh1)):
            assert torch.equal(got[r], want)
        assert torch.equal(stats[:, r], st1)

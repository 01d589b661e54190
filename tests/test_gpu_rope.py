"""svdq_rope against float64 (MI355X only); the bound is derived in
block_reference.py."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import block_reference as R

pytestmark = pytest.mark.gpu


def _inputs(B, L, H, Hk, D, pairs, dtype, seed, pos="int32", shared=True, far=1000):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    qk = torch.randn(B, L, H + Hk, D, device="cuda", generator=gen).to(dtype)
    shape = (L, len(pairs)) if shared else (B, L, len(pairs))
    p = torch.randint(-far // 2, far, shape, device="cuda", generator=gen, dtype=torch.int32)
    if pos == "fp32":
        p = p.float() * 0.37
    return qk[:, :, :H], (qk[:, :, H:] if Hk else None), p, S.rope_frequencies(pairs, 10000.0)


@pytest.mark.parametrize("B,L,H,Hk,D,pairs,dtype,interleaved,inverse,pos,shared,far", [
    (1, 1, 1, 0, 8, [1], torch.bfloat16, True, False, "int32", True, 10),
    (1, 1, 24, 24, 128, [8, 28, 28], torch.bfloat16, True, False, "int32", True, 1000),
    (2, 37, 3, 1, 72, [3, 5, 11], torch.bfloat16, True, True, "fp32", False, 1000),
    (2, 65, 5, 2, 80, [8, 12, 12], torch.float32, False, True, "fp32", True, 3000),
    (1, 130, 4, 4, 128, [16, 24, 24], torch.float16, False, False, "int32", False, 1 << 30),
    (3, 9, 2, 7, 256, [32, 32, 32, 32], torch.float32, True, False, "int32", False, 1 << 24),
    (1, 1000, 24, 8, 64, [32], torch.float16, True, True, "fp32", True, 100000),
    (1, 6, 3, 3, 40, [0, 0, 8], torch.bfloat16, False, False, "int32", True, 100),
])
def test_against_float64(B, L, H, Hk, D, pairs, dtype, interleaved, inverse, pos, shared, far):
    q, k, p, f = _inputs(B, L, H, Hk, D, pairs, dtype, L + D, pos, shared, far)
    got = S.rope(q, k, p, f, pairs, interleaved=interleaved, inverse=inverse)
    for g, x in zip(got, (q, k)):
        if x is None:
            assert g is None
        else:
            R.check(g, R.rope(x, p, f, pairs, interleaved, inverse), "rope")


@pytest.mark.parametrize("interleaved", [False, True])
def test_strides_in_place_and_passing_through(interleaved):
    """Slices of a joint projection turned in place, heads before tokens; what
    lies behind the pairs keeps its bits (NaN among them), and the values in v's
    place theirs."""
    B, L, H, D, pairs = 2, 51, 6, 96, [8, 16]
    gen = torch.Generator(device="cuda").manual_seed(4)
    qkv = torch.randn(B, L, 3, H, D, device="cuda", generator=gen).bfloat16()
    qkv[..., 49:] = float("nan")
    p, f = torch.arange(2 * L, device="cuda", dtype=torch.int32).view(L, 2), S.rope_frequencies(pairs)
    want = S.rope(qkv[:, :, 0].contiguous(), qkv[:, :, 1].contiguous(), p, f, pairs, interleaved)
    turned = [torch.empty(B, H, L, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in range(2)]
    S.rope(qkv[:, :, 0], qkv[:, :, 1], p, f, pairs, interleaved, q_out=turned[0], k_out=turned[1])
    v = qkv[:, :, 2].clone()
    got = S.rope(qkv[:, :, 0], qkv[:, :, 1], p, f, pairs, interleaved, q_out=qkv[:, :, 0], k_out=qkv[:, :, 1])
    for a, b, c in zip(got, want, turned):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(c.view(torch.int16), b.view(torch.int16))
    assert torch.equal(qkv[:, :, 2].view(torch.int16), v.view(torch.int16))
    assert bool(got[0][..., 49:].isnan().all()) and bool(got[0][..., :48].isfinite().all())


def test_gradient_is_the_inverse_turn():
    """dq = R^T dy: <rope(q), dy> == <q, rope(dy, inverse)>, in fp32 to its sums' rounding."""
    q, _, p, f = _inputs(1, 64, 4, 0, 64, [16, 16], torch.float32, 1)
    dy = torch.randn_like(q)
    y, _ = S.rope(q, None, p, f, [16, 16])
    dq, _ = S.rope(dy, None, p, f, [16, 16], inverse=True)
    a, b = (y.double() * dy.double()).sum(), (q.double() * dq.double()).sum()
    assert abs(float(a - b)) <= 16 * R.U * float((y.double() * dy.double()).abs().sum() + (q.double() * dq.double()).abs().sum())


def test_stream_graph_and_refusals():
    pairs = [8, 28, 28]
    q, k, p, f = _inputs(1, 100, 24, 24, 128, pairs, torch.bfloat16, 9)
    want = S.rope(q, k, p, f, pairs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = S.rope(q, k, p, f, pairs, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = S.rope(q, k, p, f, pairs)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    with pytest.raises(ValueError, match="freqs"):
        S.rope(q, k, p, f[:10], pairs)
    with pytest.raises(ValueError, match="positions"):
        S.rope(q, k, p[:50], f, pairs)
    with pytest.raises(ValueError, match="k:"):
        S.rope(q, k[:, :50], p, f, pairs)
    with pytest.raises(S.SvdqError):
        S.rope(q, k, p, f, pairs, q_out=q[:, :, :1].expand(-1, -1, 24, -1))
    assert S.rope(q[:, :0], k[:, :0], p[:0], f, pairs)[0].shape == (1, 0, 24, 128)

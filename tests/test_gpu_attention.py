"""svdq_attention_forward and _backward against float64 (MI355X only); the
bounds are derived in block_reference.py."""
import math

import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import block_reference as R

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def _inputs(B, Lq, Lk, H, Hk, D, dtype, seed, spread=1.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = (spread * torch.randn(B, Lq, H, D, device="cuda", generator=gen)).to(dtype)
    k, v = (torch.randn(B, Lk, Hk, D, device="cuda", generator=gen).to(dtype) for _ in range(2))
    dout = torch.randn(B, Lq, H, D, device="cuda", generator=gen).to(dtype)
    return q, k, v, dout


def _mask(B, Lk, seed, keep=0.6):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(B, Lk, device="cuda", generator=gen) < keep


def _run(q, k, v, dout, mask, causal, scale=None, check=True):
    o, lse = S.attention_forward(q, k, v, key_mask=mask, causal=causal, scale=scale)
    grads = S.attention_backward(dout, q, k, v, o, lse, key_mask=mask, causal=causal, scale=scale)
    if check:
        sc = scale if scale is not None else q.shape[3] ** -0.5
        ref = R.attention(q, k, v, mask, causal, sc)
        R.check(o, ref["o"], "o")
        R.check(lse, ref["lse"], "lse")
        ref = R.attention(q, k, v, mask, causal, sc, (dout, o, lse))
        for name, g in zip(("dq", "dk", "dv"), grads):
            R.check(g, ref[name], name)
    return (o, lse) + tuple(grads)


@pytest.mark.parametrize("B,Lq,Lk,H,Hk,D,dtype,causal,masked", [
    (1, 1, 1, 1, 1, 8, BF, False, False),
    (1, 1, 1, 1, 1, 128, HF, True, False),
    (1, 1, 500, 6, 2, 32, BF, False, True),
    (1, 70, 200, 4, 2, 8, BF, False, True),
    (2, 90, 150, 4, 1, 24, HF, True, True),
    (1, 310, 5, 9, 9, 16, BF, False, False),
    (1, 2000, 300, 24, 24, 32, HF, True, False),     # whole units in workgroups of eight waves
    (1, 40, 3000, 2, 2, 32, BF, True, False),
    (2, 1, 77, 4, 2, 64, BF, False, True),
    (1, 33, 31, 2, 1, 40, HF, False, False),
    (1, 64, 64, 2, 2, 64, BF, False, False),
    (1, 64, 64, 2, 2, 128, BF, True, False),
    (2, 65, 63, 3, 3, 72, HF, True, True),
    (1, 127, 129, 4, 1, 128, BF, True, False),
    (1, 128, 300, 6, 2, 96, HF, False, True),
    (2, 200, 130, 3, 1, 128, BF, True, True),       # the first queries see no key
    (1, 257, 513, 5, 5, 120, HF, True, False),
    (1, 1003, 77, 3, 3, 64, BF, False, True),        # few keys: their gradients' rows in parts
    (3, 5, 1000, 8, 2, 128, HF, True, True),         # few rows: the keys in parts
    (1, 1, 4100, 32, 8, 128, BF, True, False),
    (1, 700, 700, 2, 2, 16, HF, False, False),
    (4, 130, 70, 24, 24, 128, BF, False, True),
    (1, 300, 260, 64, 1, 64, BF, True, False),       # all heads share one key head
    (22, 150, 290, 12, 6, 96, BF, True, True),       # many short units: workgroups of four waves
    (13, 300, 300, 20, 20, 64, HF, False, True),
    (20, 290, 140, 14, 14, 128, HF, True, False),
    (15, 140, 270, 18, 18, 24, BF, False, False),
])
def test_against_float64(B, Lq, Lk, H, Hk, D, dtype, causal, masked):
    q, k, v, dout = _inputs(B, Lq, Lk, H, Hk, D, dtype, Lq + Lk)
    mask = _mask(B, Lk, 1) if masked else None
    a = _run(q, k, v, dout, mask, causal)
    again = _run(q, k, v, dout, mask, causal, check=False)
    assert all(torch.equal(x, y) for x, y in zip(a, again))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_without_keys(D, dtype):
    """A sample whose mask leaves nothing, and queries before the first key,
    whatever their q and dout hold."""
    B, Lq, Lk, H = 3, 90, 50, 2
    q, k, v, dout = _inputs(B, Lq, Lk, H, H, D, dtype, 5)
    mask = _mask(B, Lk, 2)
    mask[1] = False
    mask[2, :20] = False   # with causal: queries up to 40 + 19 see nothing
    for causal in (False, True):
        q1, dout1 = q.clone(), dout.clone()
        if causal:
            q1[:, :40], dout1[:, :40] = math.nan, math.inf
            q1[2, 40:60], dout1[2, 40:60] = math.inf, math.nan
        o, lse, dq, dk, dv = _run(q1, k, v, dout1, mask, causal)
        assert not bool(o[1].any()) and bool((lse[1] == -math.inf).all())
        assert not bool(dq[1].any()) and not bool(dk[1].any()) and not bool(dv[1].any())
        if causal:
            assert not bool(o[:, :40].any()) and not bool(dq[:, :40].any()) and not bool(dq[2, :60].any())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_what_stands_in_masked_places_does_not_count(dtype):
    B, Lq, Lk, H, Hk, D = 2, 150, 200, 4, 2, 128
    q, k, v, dout = _inputs(B, Lq, Lk, H, Hk, D, dtype, 6)
    mask = _mask(B, Lk, 3, 0.5)
    mask[0, 64:128] = False   # a whole tile
    want = _run(q, k, v, dout, mask, False)
    for bad in (math.nan, math.inf, torch.finfo(dtype).min):
        k1, v1 = k.clone(), v.clone()
        k1[~mask], v1[~mask] = bad, bad
        got = _run(q, k1, v1, dout, mask, False, check=False)
        assert all(torch.equal(x, y) for x, y in zip(got, want)), bad
    as_bytes = mask.to(torch.uint8) * 2   # any value that is not zero
    got = _run(q, k, v, dout, as_bytes, False, check=False)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_not_finite_values_show():
    q, k, v, dout = _inputs(1, 100, 100, 2, 2, 64, BF, 7)
    q[0, 7, 0, 3] = math.nan
    o, lse, dq, dk, dv = _run(q, k, v, dout, None, False, check=False)
    assert bool(o[0, 7, 0].isnan().all()) and bool(lse[0, 0, 7].isnan()) and bool(dq[0, 7, 0].isnan().all())
    keep = torch.ones(100, dtype=torch.bool, device="cuda")
    keep[7] = False
    assert bool(o[0, keep].isfinite().all()) and bool(o[0, 7, 1].isfinite().all())
    v[0, 50, 1, 0] = math.inf
    o, _ = S.attention_forward(q, k, v)
    assert bool((~o[0, :, 1, 0].isfinite()).all()) and bool(o[0, :, 1, 1:].isfinite().all())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_peaked_flat_and_rising_scores(dtype):
    """Scores of hundreds (a row is one key), equal scores, and scores that
    rise along the keys, so that the maximum moves at every tile."""
    B, Lq, Lk, H, D = 1, 70, 400, 2, 64
    q, k, v, dout = _inputs(B, Lq, Lk, H, H, D, dtype, 8, spread=40.0)
    _run(q, k, v, dout, None, False, scale=0.5)
    _run(torch.zeros_like(q), k, v, dout, None, True)
    k = k * 0.05 + torch.linspace(-2, 2, Lk, device="cuda")[None, :, None, None].to(dtype)
    q = q.abs()
    _run(q, k.to(dtype), v, dout, None, False, scale=0.1)
    _run(q, -k.to(dtype), v, dout, None, True, scale=0.1)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("scale", [2.0 ** -64, 2.0 ** -20, 8.0])
def test_scales(scale, dtype):
    q, k, v, dout = _inputs(1, 130, 300, 2, 2, 64, dtype, 15)
    _run(q, k, v, dout, _mask(1, 300, 6), True, scale=scale)


@pytest.mark.parametrize("small", [1e-6, 1.0, 1e4])
def test_fp16_gradients_of_any_size(small):
    """Gradients far below and near the ends of fp16 (values that fp16 holds
    among their inputs): ds is scaled, so only the results' own steps show."""
    q, k, v, dout = _inputs(1, 300, 1000, 2, 1, 64, HF, 9)
    v = (v * 8).to(HF)
    dout = (dout * small).to(HF)
    _run(q, k, v, dout, None, False, scale=0.05)


@pytest.mark.parametrize("D", [24, 64, 128])
@pytest.mark.parametrize("at", range(0, 8, 2))
def test_fp16_gradients_whose_largest_inputs_stand_anywhere(at, D):
    """The scale of ds follows the largest |dout| and |v|, at whichever two of
    eight elements these stand."""
    q, k, v, dout = _inputs(2, 150, 200, 2, 1, D, HF, 14)
    few = torch.zeros(D, dtype=torch.bool, device="cuda")
    few[at::8] = few[at + 1::8] = True
    v, dout = (torch.where(few, x * 64, x * 2.0 ** -10) for x in (v, dout))
    _run(q, k, v, dout, _mask(2, 200, 5), True)


def test_strides_and_orders():
    """Slices of a joint projection, heads before tokens, outputs of other
    orders, rows and heads apart; what lies between stays."""
    B, L, H, D = 2, 140, 3, 72
    gen = torch.Generator(device="cuda").manual_seed(10)
    qkv = torch.randn(B, L, 3, H, D, device="cuda", generator=gen).to(BF)
    dout = torch.randn(B, H, L, D, device="cuda", generator=gen).to(BF).transpose(1, 2)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    want = _run(q.contiguous(), k.contiguous(), v.contiguous(), dout.contiguous(), None, True)
    out = torch.full((B, L + 1, H, D + 8), 7.0, dtype=BF, device="cuda")
    o, lse = S.attention_forward(q, k, v, causal=True, out=out[:, 1:, :, 8:])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert bool((out[:, 0] == 7).all()) and bool((out[..., :8] == 7).all())
    dqkv = torch.full((B, 3, H, L, D), 5.0, dtype=BF, device="cuda")
    dq, dk, dv = (dqkv[:, i].transpose(1, 2) for i in range(3))
    got = S.attention_backward(dout, q, k, v, o, lse, causal=True, dq=dq, dk=dk, dv=dv)
    assert all(torch.equal(a, b) for a, b in zip(got, want[2:]))
    # keys of one sample shared by all (a batch stride of zero)
    ks, vs = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
    o1, _ = S.attention_forward(q, ks, vs)
    o2, _ = S.attention_forward(q, ks.contiguous(), vs.contiguous())
    assert torch.equal(o1, o2)


def test_zero_lengths():
    q, k, v, dout = _inputs(2, 5, 0, 2, 1, 64, HF, 11)
    o, lse, dq, dk, dv = _run(q, k, v, dout, None, False, check=False)
    assert not bool(o.any()) and bool((lse == -math.inf).all()) and not bool(dq.any()) and dk.shape == (2, 0, 1, 64)
    q, k, v, dout = _inputs(2, 0, 300, 2, 1, 64, HF, 11)
    o, lse, dq, dk, dv = _run(q, k, v, dout, None, True, check=False)
    assert o.shape == (2, 0, 2, 64) and not bool(dk.any()) and not bool(dv.any())


@pytest.mark.parametrize("Lq,Lk", [(300, 300), (2, 1500)])
def test_streams_graphs_and_workspaces(Lq, Lk):
    q, k, v, dout = _inputs(1, Lq, Lk, 4, 2, 128, HF, 12)
    mask = _mask(1, Lk, 4)
    want = _run(q, k, v, dout, mask, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = S.attention_forward(q, k, v, key_mask=mask, causal=True, stream=side)
    got = S.attention_backward(dout, q, k, v, o, lse, key_mask=mask, causal=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((o, lse) + got, want))
    # one workspace for two captured graphs that are replayed in turn, full of garbage between
    n = max(S.attention_workspace_bytes(1, Lq, Lk, 4, 2, 128, HF), S.attention_backward_workspace_bytes(1, Lq, Lk, 4, 2, 128, HF))
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, lse = S.attention_forward(q, k, v, key_mask=mask, causal=True, workspace=ws)
            outs.append((o, lse) + S.attention_backward(dout, q, k, v, o, lse, key_mask=mask, causal=True, workspace=ws))
        graphs.append(graph)
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            for t in out:
                t.zero_()
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_python_refusals():
    q, k, v, dout = _inputs(1, 10, 10, 2, 2, 64, BF, 13)
    o, lse = S.attention_forward(q, k, v)
    with pytest.raises(S.SvdqError):
        S.attention_forward(q, k, v, scale=-1.0)
    with pytest.raises(S.SvdqError):
        S.attention_forward(q, k, v, out=o[:, :1].expand(-1, 10, -1, -1))
    with pytest.raises(ValueError, match="lse"):
        S.attention_backward(dout, q, k, v, o, lse.half())
    with pytest.raises(ValueError, match="o:"):
        S.attention_backward(dout, q, k, v, o[:, :5], lse)
    with pytest.raises(ValueError, match="dtype"):
        S.attention_forward(q.double(), k.double(), v.double())
    with pytest.raises(S.SvdqError):
        S.attention_forward(q.float(), k.float(), v.float())
    with pytest.raises(ValueError, match="GPU"):
        S.attention_forward(q, k.cpu(), v)
    with pytest.raises(S.SvdqError):
        S.attention_forward(q, k, v, key_mask=torch.ones(1, 10, dtype=torch.bool, device="cuda"),
                            workspace=torch.empty(0, dtype=torch.uint8, device="cuda"), scale=float("nan"))
    with pytest.warns(UserWarning, match="autograd"):
        S.attention_forward(q.clone().requires_grad_(), k, v)

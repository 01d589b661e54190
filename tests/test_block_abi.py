"""Refusals of the entry points of the gated residual, rotary positions and
attention: every check comes before a launch, so none of this needs a GPU."""
import ctypes
import math

import pytest

import bit_svdquant_diffusion_amd as S
from tests import hip_stub as H

NULL, SHAPE, FORMAT, WORKSPACE = 1, 2, 3, 4
P = 0x7f0000000000   # an aligned address that is never read
b = ctypes.byref


def residual(channels=64, dtype=0, pdtype=0, kind=0, post=0, one_plus=0, groups=1, eps=1e-6, alpha=1.0, rpg=100):
    return b(S.ResidualDesc(channels, dtype, pdtype, kind, post, one_plus, groups, eps, alpha, rpg))


def params(gate=P, weight=P, bias=P, post=None, ld=64):
    return b(S.ResidualParams(gate, weight, bias, post, ld, ld, ld, ld))


def fwd(d, x=P, ldx=64, h=P, ldh=64, p=None, M=4, s=P, lds=64, y=P + 4096, ldy=64, st=P):
    return S.lib().svdq_residual_norm_forward(d, x, ldx, h, ldh, p, M, s, lds, y, ldy, st, None)


def bwd(d, dy=P, lddy=64, ds=P, ldds=64, s=P, lds=64, h=P, ldh=64, p=None, st=P, M=4, dx=P, lddx=64, dh=P + 4096, lddh=64,
        g=None, gd=2, ws=P, n=1 << 40):
    return S.lib().svdq_residual_norm_backward(d, dy, lddy, ds, ldds, s, lds, h, ldh, p, st, M, dx, lddx, dh, lddh, g, gd, ws, n,
                                               None)


@pytest.mark.parametrize("desc,status", [
    (dict(channels=0), SHAPE), (dict(channels=8193), SHAPE), (dict(dtype=3), FORMAT), (dict(pdtype=-1), FORMAT),
    (dict(kind=2), FORMAT), (dict(groups=0), SHAPE), (dict(rpg=0), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=math.nan), SHAPE), (dict(alpha=math.inf), SHAPE), (dict(rpg=3), SHAPE), (dict(groups=(1 << 24) + 1), SHAPE)])
def test_residual_descriptor(desc, status):
    assert fwd(residual(**desc)) == status and bwd(residual(**desc)) == status
    n = ctypes.c_size_t()
    assert S.lib().svdq_residual_norm_backward_workspace_bytes(residual(**desc), 4, b(n)) == status


def test_residual_arguments():
    assert fwd(None) == NULL and bwd(None) == NULL
    for bad, status in [(dict(x=None), NULL), (dict(h=None), NULL), (dict(s=None), NULL), (dict(y=None), NULL),
                        (dict(ldx=63), SHAPE), (dict(ldh=0), SHAPE), (dict(lds=1), SHAPE), (dict(ldy=-64), SHAPE),
                        (dict(x=P + 1), SHAPE), (dict(st=P + 2), SHAPE), (dict(M=-1), SHAPE), (dict(M=(1 << 24) + 1), SHAPE),
                        (dict(s=P + 4096), SHAPE), (dict(p=params(gate=P + 1)), SHAPE), (dict(p=params(post=P)), SHAPE)]:
        assert fwd(residual(rpg=1 << 30), **bad) == status, bad
    assert fwd(residual(groups=2), p=params(ld=10)) == SHAPE   # the stride counts with several groups
    assert fwd(residual(), M=0, x=None, h=None, s=None, y=None) == 0
    grads = b(S.ResidualGrads(P, P, P, None))
    for bad, status in [(dict(dy=None), NULL), (dict(s=None), NULL), (dict(h=None), NULL), (dict(dx=None), NULL),
                        (dict(dh=None), NULL), (dict(st=None), NULL), (dict(ldds=3), SHAPE), (dict(lddh=1), SHAPE),
                        (dict(gd=7), FORMAT), (dict(dh=P), SHAPE), (dict(g=b(S.ResidualGrads(P + 2, None, None, None))), SHAPE),
                        (dict(g=b(S.ResidualGrads(None, None, None, P))), SHAPE), (dict(M=4000, ws=None, g=grads), NULL),
                        (dict(M=4000, ws=P + 8, g=grads), SHAPE), (dict(M=4000, n=16, g=grads), WORKSPACE)]:
        assert bwd(residual(rpg=1 << 30), **bad) == status, bad
    assert bwd(residual(), M=0) == 0
    n = ctypes.c_size_t()
    f = S.lib().svdq_residual_norm_backward_workspace_bytes
    assert f(residual(), 4, None) == NULL and f(residual(rpg=4), 4, b(n)) == 0 and n.value == 0
    assert f(residual(rpg=1 << 30), 4000, b(n)) == 0 and n.value > 0
    assert f(residual(rpg=(1 << 63) - 1), 1 << 24, b(n)) == 0


def heads(p=P, batch=1 << 36, token=1024, head=128):
    return b(S.Heads(p, batch, token, head))


def rope(d=None, q=heads(), k=heads(), pos=P, pb=0, fr=P, qo=heads(), ko=heads(), **desc):
    f = dict(dtype=0, position_type=0, head_dim=128, q_heads=8, k_heads=8, axes=2, pairs=(16, 48), half=0, inverse=0, samples=2,
             tokens=100)
    f.update(desc)
    f["pairs"] = (ctypes.c_int32 * 4)(*f["pairs"])
    return S.lib().svdq_rope(b(S.RopeDesc(*[f[n] for n, _ in S.RopeDesc._fields_])), q, k, pos, pb, fr, qo, ko, None)


def test_rope_arguments():
    assert S.lib().svdq_rope(None, *[None] * 3, 0, None, None, None, None) == NULL
    for bad, status in [
            (dict(dtype=5), FORMAT), (dict(position_type=2), FORMAT), (dict(head_dim=132), SHAPE), (dict(head_dim=264), SHAPE),
            (dict(axes=0), SHAPE), (dict(axes=5), SHAPE), (dict(pairs=(32, 40)), SHAPE), (dict(pairs=(0, 0)), SHAPE),
            (dict(pairs=(-1, 3)), SHAPE), (dict(pairs=(5, 8), half=1), SHAPE), (dict(q_heads=-1), SHAPE),
            (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 22) + 1), SHAPE), (dict(samples=1 << 40), SHAPE), (dict(q=None), NULL),
            (dict(k=None), NULL), (dict(qo=None), NULL), (dict(ko=heads(p=None)), NULL), (dict(q=heads(p=P + 8)), SHAPE),
            (dict(q=heads(token=1020)), SHAPE), (dict(k=heads(head=-128)), SHAPE), (dict(qo=heads(token=1000)), SHAPE),
            (dict(qo=heads(batch=0)), SHAPE), (dict(ko=heads(head=120)), SHAPE), (dict(pos=None), NULL), (dict(fr=None), NULL),
            (dict(pos=P + 2), SHAPE), (dict(fr=P + 4), SHAPE), (dict(pb=-1), SHAPE)]:
        assert rope(**bad) == status, bad
    assert rope(tokens=0, q=None, k=None, pos=None) == 0 and rope(q_heads=0, k_heads=0, q=None, k=None) == 0


def attention(dtype=0, head_dim=128, heads=8, kv_heads=8, causal=0, scale=0.1, samples=2, queries=100, keys=100):
    return b(S.AttentionDesc(dtype, head_dim, heads, kv_heads, causal, scale, samples, queries, keys))


def afwd(d, q=heads(), k=heads(), v=heads(), mask=None, mb=0, o=heads(), lse=P, ws=P, n=1 << 50):
    return S.lib().svdq_attention_forward(d, q, k, v, mask, mb, o, lse, ws, n, None)


def abwd(d, do=heads(), q=heads(), k=heads(), v=heads(), o=heads(), lse=P, mask=None, mb=0, dq=heads(), dk=heads(), dv=heads(),
         ws=P, n=1 << 50):
    return S.lib().svdq_attention_backward(d, do, q, k, v, o, lse, mask, mb, dq, dk, dv, ws, n, None)


@pytest.mark.parametrize("desc,status", [
    (dict(dtype=2), FORMAT), (dict(dtype=-1), FORMAT), (dict(head_dim=0), SHAPE), (dict(head_dim=132), SHAPE),
    (dict(head_dim=12), SHAPE), (dict(kv_heads=0), SHAPE), (dict(kv_heads=3), SHAPE), (dict(heads=4), SHAPE),
    (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=math.nan), SHAPE), (dict(scale=math.inf), SHAPE),
    (dict(scale=2.0 ** -65), SHAPE), (dict(scale=2.0 ** 65), SHAPE),
    (dict(samples=-1), SHAPE), (dict(queries=-1), SHAPE), (dict(keys=1 << 30), SHAPE), (dict(samples=10000), SHAPE),
    (dict(kv_heads=1, queries=1 << 27), SHAPE), (dict(queries=1 << 27), SHAPE)])
def test_attention_descriptor(desc, status):
    n = ctypes.c_size_t()
    d = attention(**desc)
    assert afwd(d) == status and abwd(d) == status
    assert S.lib().svdq_attention_workspace_bytes(d, b(n)) == status
    assert S.lib().svdq_attention_backward_workspace_bytes(d, b(n)) == status


def test_attention_arguments():
    d = attention()
    assert afwd(None) == NULL and abwd(None) == NULL
    assert S.lib().svdq_attention_workspace_bytes(d, None) == NULL
    assert S.lib().svdq_attention_backward_workspace_bytes(d, None) == NULL
    bad_in = [(None, NULL), (heads(p=None), NULL), (heads(p=P + 2), SHAPE), (heads(token=100), SHAPE), (heads(batch=-8), SHAPE),
              (heads(token=1 << 25), SHAPE)]
    bad_out = bad_in + [(heads(token=512), SHAPE), (heads(batch=512), SHAPE), (heads(head=64), SHAPE)]
    for bad, status in bad_in:
        for name in ("q", "k", "v"):
            assert afwd(d, **{name: bad}) == status, (name, status)
        for name in ("do", "q", "k", "v", "o"):
            assert abwd(d, **{name: bad}) == status, (name, status)
    for bad, status in bad_out:
        assert afwd(d, o=bad) == status
        for name in ("dq", "dk", "dv"):
            assert abwd(d, **{name: bad}) == status, (name, status)
    for f in (afwd, abwd):
        assert f(d, lse=None) == NULL and f(d, lse=P + 2) == SHAPE and f(d, mask=P, mb=-1) == SHAPE
        assert f(attention(queries=1, keys=100000), ws=None) == NULL and f(attention(queries=1, keys=100000), ws=P + 8) == SHAPE
        assert f(attention(queries=1, keys=100000), n=100) == WORKSPACE
        assert f(attention(samples=0), q=None, ws=None, n=0) == 0
    assert afwd(attention(queries=0), q=None, ws=None, n=0) == 0
    # the heads of a key head within 32-bit offsets
    assert afwd(attention(kv_heads=1), q=heads(head=1 << 28)) == SHAPE


def test_scales_of_attention():
    """The forward takes scales up to 2^64, the backward up to 2^10."""
    got = H.run("""
heads = ctypes.byref(S.Heads(P, 1 << 38, 24 * 128, 128))
def both(scale):
    d = ctypes.byref(S.AttentionDesc(0, 128, 8, 8, 0, scale, 1, 300, 300))
    return [S.lib().svdq_attention_forward(d, heads, heads, heads, None, 0, heads, P, P, 1 << 40, None),
            S.lib().svdq_attention_backward(d, heads, heads, heads, heads, heads, P, None, 0, heads, heads, heads, P, 1 << 40, None)]
result = [both(2.0 ** e) for e in (-65, -64, 10, 11, 64, 65)]
""")
    assert got == [[SHAPE, SHAPE], [0, 0], [0, 0], [0, SHAPE], [0, SHAPE], [SHAPE, SHAPE]]


def test_launches_and_workspaces():
    """Which kernels a call launches (over a stand-in for the runtime): grids
    within a dimension's limit at the largest sizes, a join where there are
    few rows."""
    got = H.run("""
result = []
b = ctypes.byref
def h(): return b(S.Heads(P, 1 << 38, 24 * 128, 128))
def one(dtype, samples, queries, keys, heads, kv, causal=0):
    d = b(S.AttentionDesc(dtype, 128, heads, kv, causal, 0.1, samples, queries, keys))
    n = ctypes.c_size_t()
    sizes = []
    S.lib().svdq_attention_workspace_bytes(d, b(n)); sizes.append(n.value)
    st = [S.lib().svdq_attention_forward(d, h(), h(), h(), None, 0, h(), P, P, n.value, None)]
    f = launches()
    S.lib().svdq_attention_backward_workspace_bytes(d, b(n)); sizes.append(n.value)
    st.append(S.lib().svdq_attention_backward(d, h(), h(), h(), h(), h(), P, None, 0, h(), h(), h(), P, n.value, None))
    return [st, sizes, f, launches()]
for case in [(0, 1, 1, 1, 8, 8), (0, 1, 1, 65536, 8, 2), (1, 2, 4096, 77, 8, 8), (0, 1, 4608, 4608, 24, 24), (0, 1, 5, 0, 8, 8),
             (0, 1, 0, 5, 8, 8), (1, 16, 1 << 20, 1 << 22, 8, 8), (0, 1, 1 << 26, 1 << 26, 8, 8)]:
    result.append(one(*case))
""")
    for st, sizes, f, g in got:
        assert st == [0, 0]
        for name, grid, block in f + g:
            assert all(0 < x * y < 1 << 32 for x, y in zip(grid, block)) and grid[1] < 1 << 16 and grid[2] < 1 << 16, (name, grid)
    # (a call without queries launches no forward; a shared unit's parts are joined)
    assert [len(f) for _, _, f, _ in got] == [1, 2, 1, 1, 1, 0, 1, 1]
    assert all("join" in f[1][0] for _, _, f, _ in got if len(f) == 2)
    assert got[0][1][0] == 0 and got[1][1][0] >= 8 * 129 * 4 * 64 and got[2][1][0] == 0


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x, q = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        S.residual_norm_forward(x, x)
    with pytest.raises(ValueError, match="GPU"):
        S.rope(q, None, x, x, [32])
    with pytest.raises(ValueError, match="GPU"):
        S.attention_forward(q, q, q)
    with pytest.raises(ValueError, match="kind"):
        S._residual_setup(64, 4, torch.bfloat16, (None,) * 4, "batch", False, 1.0, 1e-6, False, None)
    with pytest.raises(ValueError, match="gate"):
        S._residual_setup(64, 4, torch.bfloat16, (torch.ones(63), None, None, None), "rms", False, 1.0, 1e-6, False, None)
    with pytest.raises(ValueError, match="post_weight"):
        S._residual_setup(64, 4, torch.bfloat16, (torch.ones(64), None, None, torch.ones(64).half()), "rms", True, 1.0, 1e-6,
                          False, None)
    with pytest.raises(ValueError, match="contiguous along the head"):
        S._heads(q.transpose(2, 3), "q", (1, 4, 64, 2), q.dtype)
    with pytest.raises(ValueError, match="shape"):
        S._heads(q, "o", (1, 4, 2, 32), q.dtype)
    with pytest.raises(ValueError, match="k, v"):
        S._attention_setup(q, q[..., :32], q, None, False, None)
    with pytest.raises(ValueError, match="key_mask"):
        S._attention_setup(q, q, q, torch.ones(1, 5, dtype=torch.bool), False, None)
    with pytest.raises(ValueError, match="key_mask"):
        S._attention_setup(q, q, q, torch.ones(1, 4), False, None)
    with pytest.raises(S.SvdqError):
        S._attention_setup(q, q, q, None, False, -1.0)


def test_rope_frequencies():
    torch = pytest.importorskip("torch")
    f = S.rope_frequencies([4, 2], 100.0, device="cpu")
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1, 100 ** -0.25, 0.1, 100 ** -0.75, 1, 0.1]).double())
    f = S.rope_frequencies([4, 0, 2], 100.0, shared=True, device="cpu")
    assert torch.allclose(f, 100.0 ** -(torch.arange(6).double() / 6))


def test_numbers_that_change_in_place():
    """alpha and eps may be any number, also one that is written in place
    between two calls: a descriptor is kept by value."""
    torch = pytest.importorskip("torch")

    def residual_of(alpha, eps):
        d = S._residual_setup(64, 4, torch.bfloat16, (None,) * 4, "rms", False, alpha, eps, False, None)[0]
        return ctypes.cast(d, ctypes.POINTER(S.ResidualDesc)).contents

    def norm_of(eps):
        d = S._norm_params(64, None, None, False, eps, None, 4, torch.bfloat16)[0]
        return ctypes.cast(d, ctypes.POINTER(S.NormDesc)).contents

    alpha, eps = torch.tensor(0.5), torch.tensor(0.25)
    assert residual_of(alpha, eps).alpha == 0.5 and residual_of(alpha, eps).eps == 0.25 and norm_of(eps).eps == 0.25
    alpha.fill_(2.0)
    eps.fill_(1.0)
    assert residual_of(alpha, eps).alpha == 2.0 and residual_of(alpha, eps).eps == 1.0 and norm_of(eps).eps == 1.0
    with pytest.raises((TypeError, ValueError)):
        residual_of("a", 0.0)

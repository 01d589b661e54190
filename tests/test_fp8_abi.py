"""Refusals of the layer norm's and the FP8 linear's entry points: every check
comes before a launch, so none of this needs a GPU."""
import ctypes

import pytest

import bit_svdquant_diffusion_amd as S

NULL, SHAPE, FORMAT, WORKSPACE, DEVICE = 1, 2, 3, 4, 6
P = 0x7f0000000000   # an aligned address that is never read


def norm(channels=64, dtype=0, pdtype=0, one_plus=0, groups=1, eps=1e-6, rpg=100):
    return ctypes.byref(S.NormDesc(channels, dtype, pdtype, one_plus, groups, eps, rpg))


def fwd(d, x=P, ldx=64, w=P, ldw=64, b=P, ldb=64, M=4, y=P, ldy=64, mean=P, rstd=P):
    return S.lib().svdq_layer_norm_forward(d, x, ldx, w, ldw, b, ldb, M, y, ldy, mean, rstd, None)


def bwd(d, dy=P, lddy=64, x=P, ldx=64, w=P, ldw=64, mean=P, rstd=P, M=4, dx=P, lddx=64, dw=P, db=P, gd=2, ws=P, n=1 << 40):
    return S.lib().svdq_layer_norm_backward(d, dy, lddy, x, ldx, w, ldw, mean, rstd, M, dx, lddx, dw, db, gd, ws, n, None)


@pytest.mark.parametrize("desc,status", [
    (dict(channels=0), SHAPE), (dict(channels=16385), SHAPE), (dict(dtype=3), FORMAT), (dict(pdtype=-1), FORMAT),
    (dict(groups=0), SHAPE), (dict(rpg=0), SHAPE), (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(rpg=3), SHAPE),                     # four rows, one group of three
    (dict(groups=(1 << 24) + 1), SHAPE)])
def test_norm_descriptor(desc, status):
    assert fwd(norm(**desc)) == status and bwd(norm(**desc)) == status
    n = ctypes.c_size_t()
    assert S.lib().svdq_layer_norm_backward_workspace_bytes(norm(**desc), 4, ctypes.byref(n)) == status


def test_norm_arguments():
    assert fwd(None) == NULL and bwd(None) == NULL
    for bad, status in [(dict(x=None), NULL), (dict(y=None), NULL), (dict(ldx=63), SHAPE), (dict(ldy=0), SHAPE),
                        (dict(x=P + 1), SHAPE), (dict(w=P + 1), SHAPE), (dict(mean=P + 2), SHAPE), (dict(M=-1), SHAPE),
                        (dict(M=(1 << 24) + 1), SHAPE)]:
        assert fwd(norm(rpg=1 << 30), **bad) == status, bad
    assert fwd(norm(groups=2), ldw=10) == SHAPE      # the stride counts with several groups
    assert fwd(norm(), M=0, x=None, y=None) == 0
    for bad, status in [(dict(dy=None), NULL), (dict(x=None), NULL), (dict(dx=None), NULL), (dict(mean=None), NULL),
                        (dict(rstd=None), NULL), (dict(gd=5), FORMAT), (dict(lddy=1), SHAPE), (dict(lddx=1), SHAPE),
                        (dict(dw=P + 2), SHAPE), (dict(M=4000, ws=None), NULL), (dict(M=4000, ws=P + 8), SHAPE),
                        (dict(M=4000, n=16), WORKSPACE)]:
        assert bwd(norm(rpg=1 << 30), **bad) == status, bad
    assert bwd(norm(), M=0, dw=None, db=None) == 0
    n = ctypes.c_size_t()
    assert S.lib().svdq_layer_norm_backward_workspace_bytes(norm(), 4, None) == NULL
    assert S.lib().svdq_layer_norm_backward_workspace_bytes(norm(rpg=4), 4, ctypes.byref(n)) == 0 and n.value == 0


def fp8(K=256, N=128):
    return ctypes.byref(S.Fp8Desc(K, N))


def packed(**over):
    f = dict(q=P, s=P, qt=P, st=P, bias=P)
    f.update(over)
    return ctypes.byref(S.Fp8Packed(*[f[n] for n in S.FP8_FIELDS]))


@pytest.mark.parametrize("K,N", [(0, 16), (16, 0), (24, 16), (16, 40), (65552, 16), (16, 65552), (-16, 16)])
def test_fp8_descriptor(K, N):
    L, n = S.lib(), ctypes.c_size_t()
    assert L.svdq_fp8_packed_bytes(fp8(K, N), ctypes.byref(S.Fp8Sizes())) == SHAPE
    assert L.svdq_fp8_workspace_bytes(fp8(K, N), 4, ctypes.byref(n)) == SHAPE
    assert L.svdq_fp8_forward(fp8(K, N), packed(), P, 4, P, P, 1 << 40, None) == SHAPE
    assert L.svdq_fp8_backward(fp8(K, N), packed(), P, P, 4, P, P, P, P, 1 << 40, None) == SHAPE
    assert L.svdq_fp8_pack(fp8(K, N), P, 2, packed(), None) == SHAPE


def test_fp8_sizes():
    assert S.fp8_packed_bytes(2064, 1552) == {"q": 2064 * 1552, "s": 13 * 20, "qt": 2064 * 1552, "st": 17 * 16,
                                              "bias": 3104}
    assert S.fp8_workspace_bytes(256, 128, 16) == 0 and S.fp8_workspace_bytes(256, 128, 0) == 0
    assert S.fp8_workspace_bytes(256, 128, 17) >= 17 * 256 + 17 * 4
    assert S.fp8_norm_workspace_bytes(256, 128, 1) >= 256 + 4
    assert S.fp8_backward_workspace_bytes(256, 128, 5) >= 5 * 128 + 256 * 128 + 128 * 128 + 128 * 4


def test_fp8_forward_arguments():
    f = lambda p=packed(), x=P, M=100, y=P, ws=P, n=1 << 40: S.lib().svdq_fp8_forward(fp8(), p, x, M, y, ws, n, None)  # noqa: E731
    for bad, status in [(dict(p=None), NULL), (dict(p=packed(q=None)), NULL), (dict(p=packed(s=None)), NULL),
                        (dict(p=packed(q=P + 8)), SHAPE), (dict(p=packed(bias=P + 2)), SHAPE), (dict(x=None), NULL),
                        (dict(y=None), NULL), (dict(x=P + 8), SHAPE), (dict(y=P + 2), SHAPE), (dict(ws=None), NULL),
                        (dict(ws=P + 4), SHAPE), (dict(n=100), WORKSPACE), (dict(M=-1), SHAPE),
                        (dict(M=(1 << 24) + 1), SHAPE)]:
        assert f(**bad) == status, bad
    assert f(M=0, x=None, y=None, ws=None, n=0) == 0
    L = S.lib()
    nf = lambda d, M=100, p=packed(), w=P, ld=256, n=1 << 40: L.svdq_fp8_norm_forward(d, w, ld, P, ld, fp8(), p, P, M, P, P, P, P, n, None)  # noqa: E731
    assert nf(norm(channels=128)) == SHAPE and nf(norm(channels=256, dtype=2)) == FORMAT
    assert nf(norm(channels=256), n=10) == WORKSPACE and nf(norm(channels=256), p=packed(q=None)) == NULL
    assert nf(norm(channels=256, groups=2), ld=100) == SHAPE and nf(norm(channels=256), w=P + 1) == SHAPE
    assert nf(norm(channels=256, rpg=50)) == SHAPE


def test_fp8_backward_and_pack_arguments():
    L = S.lib()
    f = lambda p=packed(), x=P, dy=P, M=100, dx=P, dw=P, db=P, ws=P, n=1 << 40: L.svdq_fp8_backward(  # noqa: E731
        fp8(), p, x, dy, M, dx, dw, db, ws, n, None)
    for bad, status in [(dict(p=packed(qt=None)), NULL), (dict(p=packed(st=None)), NULL),
                        (dict(p=None), NULL), (dict(dy=None), NULL), (dict(x=None), NULL), (dict(ws=None), NULL),
                        (dict(n=1), WORKSPACE), (dict(dx=P + 8), SHAPE), (dict(dw=P + 4), SHAPE), (dict(ws=P + 8), SHAPE),
                        (dict(M=(1 << 20) + 1), SHAPE)]:
        assert f(**bad) == status, bad
    assert f(dx=None, dw=None, db=None) == 0
    assert L.svdq_fp8_pack(fp8(), None, 2, packed(), None) == NULL
    assert L.svdq_fp8_pack(fp8(), P, 2, packed(qt=None), None) == NULL
    assert L.svdq_fp8_pack(fp8(), P, 7, packed(), None) == FORMAT
    assert L.svdq_fp8_pack(fp8(), P + 4, 2, packed(), None) == SHAPE
    n = ctypes.c_size_t()
    assert L.svdq_fp8_backward_workspace_bytes(fp8(), (1 << 20) + 1, ctypes.byref(n)) == SHAPE
    assert L.svdq_fp8_quantize(P, 4, 24, P, P, None) == SHAPE and L.svdq_fp8_quantize(None, 4, 32, P, P, None) == NULL


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        S.layer_norm_forward(x)
    with pytest.raises(ValueError, match="GPU"):
        S.fp8_forward(64, 64, {"q": x}, x)
    with pytest.raises(ValueError, match="dtype"):
        S._dt(torch.float64)
    with pytest.raises(ValueError):
        S._rows(x.t(), "x")
    with pytest.raises(ValueError):
        S._norm_params(64, torch.ones(63), None, False, 1e-6, None, 4, torch.bfloat16)
    with pytest.raises(ValueError):
        S._fp8_struct(64, 64, {"q": torch.zeros(10, dtype=torch.uint8)})

"""The set-up of a device (no GPU): attention kernels that refuse their
attributes stop attention's calls and no others, and the other way round."""
import pytest

from tests import hip_stub as H

_CALLS = """
heads = ctypes.byref(S.Heads(P, 1 << 30, 1024, 128))
ad = ctypes.byref(S.AttentionDesc(0, 128, 8, 8, 1, 0.1, 2, 100, 100))
rd = ctypes.byref(S.ResidualDesc(64, 0, 0, 0, 0, 0, 1, 1e-6, 1.0, 100))
def attention():
    return S.lib().svdq_attention_forward(ad, heads, heads, heads, None, 0, heads, P, P, 1 << 40, None)
def attention_grad():
    return S.lib().svdq_attention_backward(ad, heads, heads, heads, heads, heads, P, None, 0, heads, heads, heads, P, 1 << 40, None)
def rope():
    d = S.RopeDesc(0, 0, 128, 8, 0, 1, (ctypes.c_int32 * 4)(64), 0, 0, 2, 100)
    return S.lib().svdq_rope(ctypes.byref(d), heads, None, P, 0, P, heads, None, None)
def residual():
    return S.lib().svdq_residual_norm_forward(rd, P, 64, P, 64, None, 4, P, 64, P + 4096, 64, P, None)
def residual_grad():
    return S.lib().svdq_residual_norm_backward(rd, P, 64, P, 64, P, 64, P, 64, None, P, 4, P, 64, P + 4096, 64, None, 2, None, 0,
                                               None)
def norm():
    return S.lib().svdq_layer_norm_forward(ctypes.byref(S.NormDesc(64, 0, 0, 0, 1, 1e-6, 9)), P, 64, None, 64, None, 64, 4, P,
                                           64, P, P, None)
names = "attention attention_grad rope residual residual_grad norm".split()
"""
DEVICE = 6


@pytest.mark.parametrize("refused,stopped", [("", set()), ("attn_fwd", {"attention", "attention_grad"}),
                                             ("attn_dkv", {"attention", "attention_grad"}), ("norm_bwd", {"norm"})])
def test_attention_kernels_that_refuse_their_attributes(refused, stopped):
    got = H.run(_CALLS + f"refuse({refused!r})\nresult = {{n: [globals()[n](), len(launches())] for n in names * 2}}")
    for name, (status, n) in got.items():
        assert (status, n == 0) == ((DEVICE, True) if name in stopped else (0, False)), (name, status, n)


def test_attention_is_set_up_by_its_own_calls():
    """What attention's kernels refuse at another call's time does not count."""
    got = H.run(_CALLS + """
refuse("attn_")
result = [norm(), residual(), rope()]
refuse("nothing")
result += [attention(), attention_grad(), len(launches())]
""")
    assert got[:5] == [0] * 5 and got[5] >= 5

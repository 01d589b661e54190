"""The set-up of a device (no GPU): kernels that refuse their attributes stop
the calls that use them and no others."""
import pytest

from tests import hip_stub as H

_CALLS = """
def awq():
    return S.lib().svdq_awq_forward(ctypes.byref(S.AwqDesc(128, 64)), ctypes.byref(S.AwqPacked(P, P, P, P, P)), P, 4, P, None)
def linear():
    n = ctypes.c_size_t()
    d = S.Layer(256, 128, 16, "int4").desc
    S.lib().svdq_workspace_bytes(ctypes.byref(d), 64, ctypes.byref(n))
    return S.lib().svdq_linear_forward(ctypes.byref(d), ctypes.byref(S.Packed(*[P] * len(S.PACKED_FIELDS))), P, 64, P, P,
                                       n.value, None)
def norm():
    return S.lib().svdq_layer_norm_forward(ctypes.byref(S.NormDesc(64, 0, 0, 0, 1, 1e-6, 9)), P, 64, None, 64, None, 64, 4, P,
                                           64, P, P, None)
def norm_grad():
    return S.lib().svdq_layer_norm_backward(ctypes.byref(S.NormDesc(64, 0, 0, 0, 1, 1e-6, 9)), P, 64, P, 64, None, 64, P, P, 4,
                                            P, 64, None, None, 2, None, 0, None)
fd, fp = ctypes.byref(S.Fp8Desc(256, 128)), ctypes.byref(S.Fp8Packed(P, P, P, P, None))
def fp8():
    return S.lib().svdq_fp8_forward(fd, fp, P, 100, P + (1 << 40), P, 1 << 40, None)
def fp8_norm():
    return S.lib().svdq_fp8_norm_forward(ctypes.byref(S.NormDesc(256, 0, 0, 0, 1, 1e-6, 100)), None, 256, None, 256, fd, fp, P,
                                         100, P, P, P, P, 1 << 40, None)
def fp8_grad():
    return S.lib().svdq_fp8_backward(fd, fp, P, P, 100, P, P, P, P, 1 << 40, None)
def fp8_pack():
    return S.lib().svdq_fp8_pack(fd, P, 2, fp, None)
names = "awq linear norm norm_grad fp8 fp8_norm fp8_grad fp8_pack".split()
"""
DEVICE = 6


@pytest.mark.parametrize("refused,stopped", [("", set()), ("fp8_", {"fp8", "fp8_norm", "fp8_grad", "fp8_pack"}),
                                             ("norm_bwd", {"norm", "norm_grad", "fp8_norm"})])
def test_added_kernels_that_refuse_their_attributes(refused, stopped):
    got = H.run(_CALLS + f"refuse({refused!r})\nresult = {{n: [globals()[n](), len(launches())] for n in names * 2}}")
    for name, (status, n) in got.items():
        assert (status, n == 0) == ((DEVICE, True) if name in stopped else (0, False)), (name, status, n)

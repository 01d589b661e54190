"""Launches at the documented limits of the sizes stay within the runtime's
(fewer than 2^32 threads a dimension); no GPU."""
import pytest

from tests import hip_stub as H


@pytest.mark.parametrize("M,K", [(1 << 24, 16), (1 << 24, 3072), (1 << 24, 3088), (1 << 24, 65536), (1 << 20, 65536),
                                 (4194303, 16384), (4194305, 16384), (5, 65536)])
def test_row_quantizer(M, K):
    status, got = H.run(f"""
a = S.lib().svdq_fp8_quantize(P, {M}, {K}, P, P, None)
b = S.lib().svdq_fp8_forward(ctypes.byref(S.Fp8Desc({K}, 16)), ctypes.byref(S.Fp8Packed(P, P, None, None, None)), P, {M},
                             P + (1 << 45), P, 1 << 60, None)
l = launches()
result = [[a, b], [s for s in l if "quant_rows" in s[0]]]
""")
    assert status == [0, 0]
    need = M * -(-(-(-K // 128) * 128) // 1024)   # a wave each
    for _, grid, block in got:
        waves = grid[0] * grid[1] * grid[2] * block[0] // 64
        assert need <= waves and waves - need < 4 * (1 << 20)


@pytest.mark.parametrize("groups,rpg,M,C,params", [(1 << 24, 1, 1000, 4096, False), (1 << 24, 1, 1 << 24, 16384, False),
                                                   (1 << 24, 1, 1000, 2048, True), (1 << 23, 2, 1 << 24, 16384, True),
                                                   (1 << 20, 1, 1 << 20, 16384, True), (1000, 1, 7, 64, True)])
@pytest.mark.parametrize("dtype", [0, 2])
def test_norm_gradient_of_many_groups(groups, rpg, M, C, params, dtype):
    status, got = H.run(f"""
n = S.NormDesc({C}, {dtype}, 2, 0, {groups}, 0.0, {rpg})
out = P if {params} else None
st = S.lib().svdq_layer_norm_backward(ctypes.byref(n), P, {C}, P, {C}, None, {C}, P, P, {M}, P, {C}, out, out, 2, P, 1 << 60,
                                      None)
result = [st, launches()]
""")
    assert status == 0 and len(got) == 1
    _, grid, block = got[0]
    assert groups <= grid[0] * grid[1] * grid[2] < groups + (1 << 20)

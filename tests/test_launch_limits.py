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

"""Which kernels the FP8 products and the large inputs take (no GPU): the
cases that the GPU tests check stay on the kernels that they are there for."""
import re

import pytest

from tests import fp8_cases as C
from tests import hip_stub as H

_CALL = """
W = P + (1 << 45)
def forward(M, K, N):
    d, p = ctypes.byref(S.Fp8Desc(K, N)), ctypes.byref(S.Fp8Packed(P, P, P, P, P))
    assert S.lib().svdq_fp8_forward(d, p, P, M, W, P, 1 << 44, None) == 0
    return launches()
def backward(M, K, N):
    d, p = ctypes.byref(S.Fp8Desc(K, N)), ctypes.byref(S.Fp8Packed(P, P, P, P, P))
    assert S.lib().svdq_fp8_backward(d, p, P, P, M, None, W, None, P, 1 << 44, None) == 0
    return launches()
"""


def _product(launches):
    """((tile), rows of B have scales, workgroups) of the product among launches"""
    name, grid, _ = next(x for x in launches if "fp8_gemm_kernel" in x[0])
    m = re.search(r"fp8_gemm_kernelILi(\d+)ELi(\d+)ELi2ELi2ELb([01])E", name)
    return (int(m[1]), int(m[2])), m[3] == "1", grid[0]


@pytest.mark.parametrize("tile", list(C.OUTPUTS))
def test_forward_tiles(tile):
    cases = [c for c in C.FORWARD if c[0] == tile]
    for (_, blocks, M, K, N), got in zip(cases, H.run(_CALL + f"result = [forward(*c[2:]) for c in {cases!r}]")):
        assert -(-K // 128) == blocks and M % tile[0] and N % tile[1]
        assert _product(got)[:2] == (tile, False)
        assert -(-M // tile[0]) * -(-N // tile[1]) > _product(got)[2]   # several tiles a workgroup


@pytest.mark.parametrize("tile", list(C.GRADIENTS))
def test_gradient_tiles(tile):
    cases = [c for c in C.BACKWARD if c[0] == tile]
    for (_, blocks, M, K, N), got in zip(cases, H.run(_CALL + f"result = [backward(*c[2:]) for c in {cases!r}]")):
        assert -(-M // 128) == blocks and N % tile[0] and K % tile[1]
        assert _product(got)[:2] == (tile, True)
        assert -(-N // tile[0]) * -(-K // tile[1]) > _product(got)[2]


def test_large_inputs_and_outputs():
    """(sizes, as no launch shows how memory is read)"""
    assert all(M * K * 2 >= 16e6 for M, K in C.QUANTIZED)
    assert any(M * (K + N) * 2 >= 16e6 for _, _, M, K, N in C.BACKWARD) and any(M * (K + N) * 2 < 16e6 for _, _, M, K, N in C.BACKWARD)
    assert all(M * c * 3 * (4 if t == "fp32" else 2) > 128e6 for M, c, t in C.NORM_GRADIENTS)
    assert any(M * N > 32e6 for _, _, M, _, N in C.FORWARD) and any(M * N < 32e6 for _, _, M, _, N in C.FORWARD)

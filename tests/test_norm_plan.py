"""The plan of the layer norm's gradients on the host (no GPU)."""
import pytest

from tests import hip_stub as H


@pytest.mark.parametrize("dtype", [0, 2])
def test_any_length_of_a_group(dtype):
    """rows_per_group up to the largest int64: groups longer than the matrix
    are one group of all rows, so the plan is that of rows_per_group == M."""
    # (in a child process: a division by zero would end this one)
    got = H.run(f"""
result = []
for M in (0, 1, 2, 3, 4, 5, 100, 9216, 1 << 24):
    row = []
    for rpg in (max(M, 1), M + 1, (1 << 62), (1 << 63) - M - 1, (1 << 63) - 1):
        n = ctypes.c_size_t()
        d = ctypes.byref(S.NormDesc(1000, {dtype}, 2, 0, 1, 1e-6, rpg))
        st = S.lib().svdq_layer_norm_backward_workspace_bytes(d, M, ctypes.byref(n))
        st2 = S.lib().svdq_layer_norm_backward(d, P, 1000, P, 1000, P, 1000, P, P, M, P, 1000, P, P, 2, P, n.value, None)
        row.append([st, n.value, st2, launches()])
    result.append(row)
""")
    for row in got:
        assert row[0][0] == 0 and row[0][2] == 0
        assert all(r == row[0] for r in row), row

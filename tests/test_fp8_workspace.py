"""Where the FP8 calls put things in their workspace (no GPU)."""
import pytest

from tests import hip_stub as H

# the product's argument: a, as, a_rows, lda, b, bs, b_rows, ldb, b_row_scales, K, bias, out, part, tickets, x
_GEMM = """
class Gemm(ctypes.Structure):
    _fields_ = [("a", ctypes.c_uint64), ("sa", ctypes.c_uint64), ("a_rows", ctypes.c_int64), ("lda", ctypes.c_int64),
                ("b", ctypes.c_uint64), ("sb", ctypes.c_uint64), ("b_rows", ctypes.c_int32), ("ldb", ctypes.c_int64),
                ("b_row_scales", ctypes.c_int32), ("K", ctypes.c_int64), ("bias", ctypes.c_uint64), ("out", ctypes.c_uint64),
                ("part", ctypes.c_uint64), ("tickets", ctypes.c_uint64), ("x", ctypes.c_uint64)]
W = P + (1 << 40)
def products():
    n = stub.stub_launches()
    kernels = [stub.stub_kernel(i).decode() for i in range(n)]
    out = [Gemm.from_buffer_copy(ctypes.string_at(first(i), ctypes.sizeof(Gemm))) for i in range(n) if "deep" in kernels[i]]
    stub.stub_clear()
    return out
def call(op, M, K, N, at):
    d, p = S.Fp8Desc(K, N), S.Fp8Packed(P, P, P, P, None)
    norm = S.NormDesc(K, 0, 0, 0, 1, 1e-6, M)
    n = S._fp8_bytes({"forward": "svdq_fp8_workspace_bytes", "norm": "svdq_fp8_norm_workspace_bytes",
                      "backward": "svdq_fp8_backward_workspace_bytes"}[op], K, N, M)
    dr, pr, L = ctypes.byref(d), ctypes.byref(p), S.lib()
    def go(size):
        if op == "forward":
            return L.svdq_fp8_forward(dr, pr, P, M, P, W + at, size, None)
        if op == "norm":
            return L.svdq_fp8_norm_forward(ctypes.byref(norm), None, K, None, K, dr, pr, P, M, P, P, P, W + at, size, None)
        return L.svdq_fp8_backward(dr, pr, P, P, M, P, P, P, W + at, size, None)
    short = go(n - 1)
    none = stub.stub_launches()
    return [short, none, go(n), n, [[g.part, g.tickets, g.a, g.a_rows, g.b_rows, g.K] for g in products()]]
"""


@pytest.mark.parametrize("op", ["forward", "norm", "backward"])
@pytest.mark.parametrize("M,K,N", [(64, 2064, 1040), (33, 12288, 64), (70, 8208, 272)])
def test_sums_of_runs_fill_whole_lines_of_their_own(op, M, K, N):
    """The sums of runs are exchanged between workgroups through the device's
    coherence point: no line of them may hold another tile's, so they start on
    256 bytes wherever the workspace starts, and end inside it."""
    if op == "backward":   # (whose dx contracts the output channels)
        K, N = N, K
    got = H.run(_GEMM + f"result = [call({op!r}, {M}, {K}, {N}, at) for at in (0, 16, 128, 240)] + [W]")
    W, joined = got.pop(), 0
    for at, (short, none, status, size, products) in zip((0, 16, 128, 240), got):
        assert (short, none, status) == (4, 0, 0)   # a byte too few is refused
        for part, tickets, a, rows, cols, k in products:
            assert W + at <= a and tickets % 4 == 0 and W + at <= tickets and tickets + 512 <= W + at + size
            if (k + 127) // 128 >= 17:   # several runs with these few tiles
                joined += 1
                assert part % 256 == 0
                assert W + at <= part and part + 4 * 64 * 64 * -(-rows // 64) * -(-cols // 64) * 2 <= W + at + size
    assert joined

"""Outputs of the FP8 linear over its inputs: refused where one kernel reads
and writes them (no GPU; the allowed ones' results in test_gpu_fp8_overlap.py)."""
from tests import hip_stub as H


def test_forward_over_its_input():
    got = H.run("""
def f(M, K, N, x, y):
    d, p = S.Fp8Desc(K, N), S.Fp8Packed(P, P, None, None, None)
    W = P + (1 << 40)   # the weight's buffers and the workspace lie elsewhere
    p.q = p.s = W
    st = S.lib().svdq_fp8_forward(ctypes.byref(d), ctypes.byref(p), x, M, y, W, 1 << 40, None)
    return [st, len(launches())]
n = 4 * 128 * 2   # bytes of x and of y
result = {
    "same": f(4, 128, 128, P, P), "one row on": f(4, 128, 128, P, P + 256), "one row back": f(4, 128, 128, P + 256, P),
    "x in a larger y": f(4, 128, 1024, P + 4096, P), "y in a larger x": f(4, 1024, 128, P, P + 4096),
    "last bytes": f(4, 128, 128, P, P + n - 16), "after": f(4, 128, 128, P, P + n), "before": f(4, 128, 128, P + n, P),
    "limit": f(16, 2944, 128, P, P), "past the limit": f(16, 3088, 128, P, P), "more tokens": f(17, 128, 128, P, P)}
""")
    SHAPE = 2
    for name in ("same", "one row on", "one row back", "x in a larger y", "y in a larger x", "last bytes", "limit"):
        assert got[name] == [SHAPE, 0], name
    assert got["after"] == [0, 1] and got["before"] == [0, 1]
    # two kernels: the first has read x before the second writes y
    assert got["past the limit"] == [0, 2] and got["more tokens"] == [0, 2]

"""The caller's choice of probabilities as two values (no GPU): which kernels
a call launches, and that its workspace is asked for with the same choice."""
import re

from tests import hip_stub as H


def test_launches():
    got = H.run("""
heads = ctypes.byref(S.Heads(P, 1 << 38, 64 * 128, 128))
def one(D, samples, queries, keys, heads_q, kv, causal, fine):
    d = ctypes.byref(S.AttentionDesc(1, D, heads_q, kv, causal, 0.1, samples, queries, keys, fine))
    n = ctypes.c_size_t()
    S.lib().svdq_attention_workspace_bytes(d, ctypes.byref(n))
    st = [S.lib().svdq_attention_forward(d, heads, heads, heads, None, 0, heads, P, P, n.value, None)]
    S.lib().svdq_attention_backward_workspace_bytes(d, ctypes.byref(n))
    st.append(S.lib().svdq_attention_backward(d, heads, heads, heads, heads, heads, P, None, 0, heads, heads, heads, P, n.value, None))
    return [D, fine, st, [l[0] for l in launches() if "attn_fwd" in l[0] or "attn_dq" in l[0] or "attn_dkv" in l[0]]]
result = [one(*c, fine) for fine in (0, 1) for c in [
    (128, 1, 4608, 4608, 24, 24, 0), (72, 2, 1531, 1601, 12, 4, 1), (64, 2, 4096, 77, 20, 20, 0), (64, 1, 300, 300, 2, 2, 1),
    (96, 22, 150, 290, 12, 6, 1), (32, 1, 2000, 300, 24, 24, 1), (128, 64, 300, 300, 12, 12, 0), (128, 1, 5, 9, 2, 2, 0)]]
""")
    for D, fine, st, names in got:
        assert st == [0, 0] and len(names) == 3
        for name in names:   # type, padded head, waves, ways, operands, parts
            dp, waves, ways, operands = map(int, re.search(r"Li(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb", name).groups())
            if fine:
                assert operands == 2 and (dp == 32 or (waves, ways) == (8, 1)), (D, name)
    assert {re.search(r"Li(\d+)ELb", n).group(1) for _, fine, _, names in got if not fine for n in names} == {"1", "2"}

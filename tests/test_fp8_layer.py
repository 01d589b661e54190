"""The FP8 layer's buffers in the binding: what a refused call leaves (no
GPU; the same on one in test_gpu_fp8_layer.py)."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S


def _buffers(K, N):
    n = S.fp8_packed_bytes(K, N)
    dev = {k: torch.zeros(n[k], dtype=torch.uint8) for k in ("q", "s", "qt", "st")}
    dev["bias"] = torch.ones(N, dtype=torch.bfloat16)
    return dev


def test_a_refused_pack_leaves_the_layer_as_it_was():
    dev = _buffers(64, 32)
    before = dict(dev)
    with pytest.raises(ValueError, match="GPU"):
        S.fp8_pack(torch.randn(32, 64), torch.zeros(32), out=dev)
    assert all(dev[k] is before[k] for k in before) and bool((dev["bias"] == 1).all())


def _layer(K, N, **over):
    n = S.fp8_packed_bytes(K, N)
    rows = {"q": N, "s": -(-N // 128), "qt": K, "st": -(-K // 128)}
    dev = {k: torch.zeros(r, n[k] // r, dtype=torch.uint8) for k, r in rows.items()}
    return dict(dev, bias=torch.zeros(N, dtype=torch.bfloat16), **over)


def test_buffers_of_the_layer_are_accepted():
    for K, N in [(16, 16), (144, 272), (2064, 1552), (1024, 128)]:
        S._fp8_struct(K, N, _layer(K, N))
        S._fp8_struct(K, N, dict(_layer(K, N), bias=None, qt=None, st=None))
        n = S.fp8_packed_bytes(K, N)   # plain bytes, as many as there must be or more
        S._fp8_struct(K, N, {k: torch.zeros(n[k] + (64 if k == "q" else 0), dtype=torch.uint8) for k in ("q", "s", "qt", "st")})
        S._fp8_struct(K, N, dict(_layer(K, N), q=_layer(K, N)["q"].view(torch.float8_e4m3fn)))


@pytest.mark.parametrize("parts", [dict(backward=False), dict(forward=False), dict()])
@pytest.mark.parametrize("K,N", [(256, 1024), (1024, 256), (272, 528), (2064, 1552)])
def test_buffers_of_another_layer_are_refused(K, N, parts):
    """Inputs and outputs exchanged, or other sizes with as many bytes."""
    for other in [(N, K), (K // 2, 2 * N) if K % 32 == 0 else (N, K), (2 * K, N // 2) if N % 32 == 0 else (N, K),
                  (K, N + 16), (K + 16, N)]:
        with pytest.raises(ValueError, match="fp8 layer"):
            S._fp8_struct(K, N, _layer(*other), **parts)


def test_each_buffer_is_checked():
    K, N = 272, 528
    good = _layer(K, N)
    for name, bad in [("q", good["qt"]), ("qt", good["q"]), ("q", good["q"].t()), ("q", good["q"][:-1]),
                      ("q", torch.zeros(N, K // 2, dtype=torch.bfloat16)), ("s", good["s"][:, :-1]), ("s", good["s"].t()),
                      ("st", good["st"][:-1]), ("bias", torch.zeros(N - 1, dtype=torch.bfloat16)),
                      ("bias", torch.zeros(N)),
                      ("q", torch.zeros(N * K - 1, dtype=torch.uint8))]:
        with pytest.raises(ValueError, match="fp8 layer"):
            S._fp8_struct(K, N, dict(good, **{name: bad}))

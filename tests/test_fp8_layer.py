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

"""FP8 calls in workspaces that start anywhere on 16 bytes (MI355X only): the
bits of a call with the allocator's alignment, and nothing written outside."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N", [(64, 2064, 1040), (33, 12288, 64), (70, 8208, 272), (1003, 272, 528)])
def test_offset_workspaces(M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M)
    w = torch.randn(N, K, device="cuda", generator=g) / K ** 0.5
    dev, back = S.fp8_pack(w), S.fp8_pack(w.t().contiguous())
    x, dy = (torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    x2 = torch.randn(M, N, device="cuda", generator=g).to(torch.bfloat16)
    calls = [(S.fp8_workspace_bytes(K, N, M), lambda ws: (S.fp8_forward(K, N, dev, x, workspace=ws),)),
             (S.fp8_norm_workspace_bytes(K, N, M), lambda ws: (S.fp8_norm_forward(K, N, dev, x, workspace=ws),)),
             # (dx contracts the K channels of dy)
             (S.fp8_backward_workspace_bytes(N, K, M), lambda ws: S.fp8_backward(N, K, back, x2, dy, workspace=ws))]
    for size, call in calls:
        want = call(None)
        for at in (0, 16, 112, 128, 240):
            room = torch.full((at + size + 512,), 0xFF, dtype=torch.uint8, device="cuda")
            got = call(room[at:at + size])
            assert all(torch.equal(p, q) for p, q in zip(got, want)), (size, at)
            assert bool((room[:at] == 0xFF).all()) and bool((room[at + size:] == 0xFF).all()), (size, at)

"""Outputs of the FP8 linear over its inputs, where that is allowed: the same
bits as into other memory (MI355X only)."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S

pytestmark = pytest.mark.gpu


def _layer(g, K, N):
    w = torch.randn(N, K, device="cuda", generator=g) / K ** 0.5
    return S.fp8_pack(w, torch.randn(N, device="cuda", generator=g))


@pytest.mark.parametrize("M,K", [(17, 128), (64, 2064), (300, 272), (16, 3088)])
def test_forward_in_place(M, K):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    dev, x = _layer(g, K, K), torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    want = S.fp8_forward(K, K, dev, x)
    assert S.fp8_forward(K, K, dev, x, y=x) is x and torch.equal(x, want)


@pytest.mark.parametrize("M", [1, 16])
def test_forward_of_a_few_tokens_in_place_is_refused(M):
    g = torch.Generator(device="cuda").manual_seed(M)
    K = 272
    dev, room = _layer(g, K, K), torch.randn(2 * M, K, device="cuda", generator=g).to(torch.bfloat16)
    x = room[:M]
    with pytest.raises(S.SvdqError):
        S.fp8_forward(K, K, dev, x, y=x)
    want = S.fp8_forward(K, K, dev, x)
    assert torch.equal(S.fp8_forward(K, K, dev, x, y=room[M:]), want)   # right behind it


@pytest.mark.parametrize("M", [1, 16, 17, 200])
def test_norm_forward_in_place(M):
    g = torch.Generator(device="cuda").manual_seed(M)
    K = 528
    dev, x = _layer(g, K, K), torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16)
    want = S.fp8_norm_forward(K, K, dev, x)
    S.fp8_norm_forward(K, K, dev, x, y=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("M,K", [(5, 272), (300, 528), (1000, 128)])
def test_backward_over_its_inputs(M, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    dev = _layer(g, K, K)
    x, dy = (torch.randn(M, K, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    want = S.fp8_backward(K, K, dev, x, dy)
    ws = torch.empty(S.fp8_backward_workspace_bytes(K, K, M), dtype=torch.uint8, device="cuda")
    for into in (0, 1):   # dx over x, over dy
        a, b = x.clone(), dy.clone()
        dw, db = torch.empty_like(want[1]), torch.empty_like(want[2])
        d, p = S._fp8_struct(K, K, dev, 0)
        S._call("svdq_fp8_backward", 0, None, d, p, a.data_ptr(), b.data_ptr(), M, (a, b)[into].data_ptr(), dw.data_ptr(),
                db.data_ptr(), ws.data_ptr(), ws.numel())
        assert all(torch.equal(p, q) for p, q in zip(((a, b)[into], dw, db), want)), into

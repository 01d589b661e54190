"""The layer norm and the FP8 linear next to torch's autograd (MI355X only):
a call outside of a graph says so, and a torch.autograd.Function made of the
calls has their gradients."""
import warnings

import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S

pytestmark = pytest.mark.gpu


def _bf16(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


def _calls(x, w, b, lin, dy, dh):
    """(call, the inputs that its gradient would belong to)"""
    _, mean, rstd = S.layer_norm_forward(x.detach(), w.detach(), b.detach())
    return {"layer_norm_forward": (lambda: S.layer_norm_forward(x, w, b)[0], (x, w, b)),
            "fp8_forward": (lambda: lin(x), (x,)),
            "fp8_norm_forward": (lambda: lin.after_norm(x, w, b), (x, w, b)),
            "layer_norm_backward": (lambda: S.layer_norm_backward(dh, x.detach(), mean, rstd, w.detach())[0], (dh,)),
            "fp8_backward": (lambda: lin.backward(x.detach(), dy)[0], (dy,))}


def test_a_call_with_inputs_that_require_grad_warns():
    g = torch.Generator(device="cuda").manual_seed(1)
    M, K, N = 20, 144, 80
    x, w, b, dy, dh = _bf16(g, M, K), _bf16(g, K), _bf16(g, K), _bf16(g, M, N), _bf16(g, M, K)
    lin = S.Fp8Linear(torch.randn(N, K, device="cuda", generator=g))
    for name, (call, inputs) in _calls(x, w, b, lin, dy, dh).items():
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            want = call()
        for t in inputs:
            t.requires_grad_(True)
            with pytest.warns(UserWarning, match=name + " records no autograd graph"):
                got = call()
            assert torch.equal(got, want) and not got.requires_grad
            with warnings.catch_warnings(), torch.no_grad():
                warnings.simplefilter("error")
                assert torch.equal(call(), want)
            t.requires_grad_(False)


class _NormLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, nw, nb, w, b, lin):
        y, mean, rstd = lin.after_norm(x, nw, nb, one_plus=True, stats=True)
        ctx.save_for_backward(x, nw, nb, mean, rstd)
        ctx.lin = lin
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, nw, nb, mean, rstd = ctx.saved_tensors
        h = S.layer_norm_forward(x, nw, nb, one_plus=True)[0]
        dh, dw, db = ctx.lin.backward(h, dy.contiguous())
        dx, dnw, dnb = S.layer_norm_backward(dh, x, mean, rstd, nw, one_plus=True)
        return dx, dnw, dnb, dw, db, None


def test_a_function_of_the_calls():
    g = torch.Generator(device="cuda").manual_seed(2)
    M, K, N = 150, 272, 144
    x, nw, nb, w, b = (t.requires_grad_(True) for t in (_bf16(g, M, K), _bf16(g, K), _bf16(g, K), _bf16(g, N, K), _bf16(g, N)))
    lin, dy = S.Fp8Linear(w, b), _bf16(g, M, N)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        _NormLinear.apply(x, nw, nb, w, b, lin).backward(dy)
    with torch.no_grad():
        h, mean, rstd = S.layer_norm_forward(x, nw, nb, one_plus=True)
        dh, dw, db = lin.backward(h, dy)
        dx, dnw, dnb = S.layer_norm_backward(dh, x, mean, rstd, nw, one_plus=True)
    for t, want in ((x, dx), (nw, dnw), (nb, dnb), (w, dw), (b, db)):
        assert torch.equal(t.grad, want)

"""svdq_residual_norm_backward with its outputs over any of its inputs, at
widths whose last vector begins a wave of its own and shares elements with the
wave before it (MI355X only): the results of a call with separate outputs."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("post,kind", [(False, "rms"), (False, "layer"), (True, "rms")])
@pytest.mark.parametrize("C,dtype", [(513, torch.bfloat16), (515, torch.float16), (519, torch.bfloat16), (1025, torch.float16),
                                     (1031, torch.bfloat16), (513, torch.float32), (515, torch.float32), (1026, torch.float32)])
def test_outputs_over_inputs(C, dtype, post, kind):
    M = 700
    gen = torch.Generator(device="cuda").manual_seed(C)
    rows = {n: torch.randn(M, C, device="cuda", generator=gen).to(dtype) for n in ("dy", "ds", "s", "h")}
    gate, weight, pw = (torch.randn(C, device="cuda", generator=gen) for _ in range(3))
    x = torch.randn(M, C, device="cuda", generator=gen).to(dtype)
    if not post:
        pw = None
    rows["s"], _, stats = S.residual_norm_forward(x, rows["h"], gate, weight, None, post_weight=pw, kind=kind)

    def call(r, dx=None, dh=None):
        return S.residual_norm_backward(r["dy"], r["s"], r["h"], stats, gate, weight, post_weight=pw, ds=r["ds"], kind=kind, dx=dx, dh=dh)
    want = call(rows)
    for a in rows:
        for b in rows:
            if a == b:
                continue
            r = {n: t.clone() for n, t in rows.items()}
            got = call(r, r[a], r[b])
            assert all(u is v or torch.equal(u, v) for u, v in zip(got, want)), (a, b)

"""The float64 references of the operators between a block's linears: their
gradients against central differences and against autograd (no GPU)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import block_reference as R


def _difference(f, x, d, at=1e-5):
    return (f(x + at * d) - f(x - at * d)) / (2 * at)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("post", [False, True])
def test_residual_norm_gradients_are_derivatives(kind, post):
    g = torch.Generator().manual_seed(1)
    rows, C, groups, rpg, alpha = 7, 11, 2, 4, 0.75
    x, h, dy, ds = (torch.randn(rows, C, generator=g, dtype=torch.float64) for _ in range(4))
    gate, w, b, pw = (torch.randn(groups, C, generator=g, dtype=torch.float64) for _ in range(4))

    def loss(x, h, gate, w, b, pw):
        hn = R.norm(h, kind, 1e-6)[0] * R.of_rows(pw, rows, rpg, 1.0) if post else h
        s = alpha * x + R.of_rows(gate, rows, rpg) * hn
        y = R.norm(s, kind, 1e-6)[0] * R.of_rows(w, rows, rpg, 1.0) + R.of_rows(b, rows, rpg)
        return (y * dy).sum() + (s * ds).sum()

    args = [x, h, gate, w, b, pw]
    hn = R.norm(h, kind, 1e-6)[0] * R.of_rows(pw, rows, rpg, 1.0) if post else h
    s = alpha * x + R.of_rows(gate, rows, rpg) * hn
    stats = []
    for v in (s, h) if post else (s,):
        _, _, m, _, r, _ = R.norm(v, kind, 1e-6)
        stats += [m, r] if kind == "layer" else [r]
    got = R.residual_norm_grad(dy, ds, s, h, stats, gate, w, pw, alpha, kind, post, True, rpg, groups, torch.float64)
    names = ["dx", "dh", "dgate", "dweight", "dbias"] + (["dpost"] if post else [])
    for i, name in enumerate(names):
        d = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        want = _difference(lambda v: loss(*args[:i], v, *args[i + 1:]), args[i], d)
        assert math.isclose(float((got[name][0] * d).sum()), float(want), rel_tol=1e-6, abs_tol=1e-7), name


@pytest.mark.parametrize("causal", [False, True])
def test_attention_gradients_are_derivatives(causal):
    g = torch.Generator().manual_seed(2)
    B, Lq, Lk, H, Hk, D, scale = 2, 5, 4, 4, 2, 8, 0.6
    q, dout = (torch.randn(B, Lq, H, D, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(B, Lk, Hk, D, generator=g, dtype=torch.float64) for _ in range(2))
    mask = torch.tensor([[True, True, False, True], [False, True, True, True]])

    def out(*qkv):
        return R.attention(*qkv, mask, causal, scale)

    o, lse = (out(q, k, v)[n][0] for n in ("o", "lse"))
    got = R.attention(q, k, v, mask, causal, scale, (dout, o, lse))
    args = [q, k, v]
    for i, name in enumerate(("dq", "dk", "dv")):
        d = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
        want = _difference(lambda t: (out(*args[:i], t, *args[i + 1:])["o"][0] * dout).sum(), args[i], d)
        assert math.isclose(float((got[name][0] * d).sum()), float(want), rel_tol=1e-6, abs_tol=1e-8), name


def test_attention_of_rows_without_keys():
    q, k = torch.ones(1, 3, 1, 8, dtype=torch.float64), torch.ones(1, 2, 1, 8, dtype=torch.float64)
    r = R.attention(q, k, k, None, True, 1.0)   # query 0 sees key -1 and before: none
    assert r["lse"][0][0, 0, 0] == -math.inf and bool((r["o"][0][0, 0] == 0).all()) and bool((r["o"][0][0, 1:] == 1).all())
    r = R.attention(q, k, k, torch.zeros(1, 2, dtype=torch.bool), False, 1.0)
    assert bool((r["o"][0] == 0).all()) and bool((r["lse"][0] == -math.inf).all())


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_turns_and_turns_back(interleaved):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 5, 3, 40, generator=g, dtype=torch.float64)
    pos = torch.randint(-1000, 100000, (2, 5, 2), generator=g, dtype=torch.int32)
    freqs = torch.rand(16, generator=g, dtype=torch.float64)
    y, _ = R.rope(x, pos, freqs, [4, 12], interleaved, False)
    back, _ = R.rope(y, pos, freqs, [4, 12], interleaved, True)
    assert torch.allclose(back, x, atol=1e-9) and torch.equal(y[..., 32:], x[..., 32:])
    assert torch.allclose(y.square().sum(-1), x.square().sum(-1))
    # a pair as a complex number
    j = 9
    u, v = (2 * j, 2 * j + 1) if interleaved else (j, j + 16)
    z = torch.complex(x[..., u], x[..., v]) * torch.exp(1j * (pos[..., 1].double() * freqs[j]))[:, :, None]
    assert torch.allclose(torch.complex(y[..., u], y[..., v]), z, atol=1e-9)

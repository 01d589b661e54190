"""svdq_residual_norm_forward and _backward against float64 (MI355X only);
the bounds are derived in block_reference.py."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import block_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _rows(gen, M, C, dtype, at=0.5):
    x = torch.randn(M, C, device="cuda", generator=gen) + at
    if C > 3:
        x[:, C // 3] *= 20
    return x.to(dtype)


def _case(M, C, dtype, pdtype, groups, one_plus, post, seed, flat=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = {n: _rows(gen, M, C, dtype) for n in ("x", "h", "dy", "ds")}
    for n in ("gate", "weight", "bias", "post"):
        p = torch.randn(groups, C, device="cuda", generator=gen) * 0.4 + (1.0 if not one_plus and n in ("weight", "post") else 0.0)
        c[n] = (p[0] if flat else p).to(pdtype)
    if not post:
        c["post"] = None
    return c


def _stat_rows(stats, kind, post):
    """[(mean or None, rstd)] of s and, with post, of h."""
    it = iter(stats)
    return [(next(it) if kind == "layer" else None, next(it)) for _ in range(2 if post else 1)]


def _check_forward(c, kind, post, one_plus, rpg, alpha, eps, s, y, stats):
    ref = R.residual_norm(c["x"], c["h"], c["gate"], c["weight"], c["bias"], c["post"], alpha, eps, kind, post, one_plus, rpg, s=s)
    R.check(s, ref["s"], "s")
    R.check(y, ref["y"], "y")
    for (mean, rstd), name in zip(_stat_rows(stats, kind, post), ("norm", "post")):
        m, em, r, er = ref[name]
        if mean is not None:
            R.check(mean, (m, em + R.U * m.abs()), f"{name} mean")
        R.check(rstd, (r, r * (er + 4 * R.U)), f"{name} rstd")


def _check_backward(c, s, stats, kind, post, one_plus, rpg, groups, alpha, got, gdtype, flat, ds):
    ref = R.residual_norm_grad(c["dy"], ds, s, c["h"], list(stats), c["gate"], c["weight"], c["post"], alpha, kind, post, one_plus,
                               rpg, groups, gdtype)
    names = ["dx", "dh", "dgate", "dweight", "dbias", "dpost"]
    for name, g in zip(names, got):
        if name == "dpost" and not post:
            assert g is None
            continue
        v, e = ref[name]
        R.check(g, (v[0], e[0]) if flat and name not in ("dx", "dh") else (v, e), name)


CASES = [
    # rows, channels, type, parameters, groups, one_plus, post, kind, alpha
    (1, 1536, "bf16", "bf16", 1, False, True, "rms", 1.0),
    (1, 1, "fp32", "fp32", 1, False, False, "layer", 1.0),
    (3, 7, "bf16", "fp32", 1, True, True, "layer", 0.5),
    (5, 33, "fp16", "fp16", 2, True, False, "rms", 1.0),
    (70, 128, "bf16", "bf16", 3, False, True, "layer", 1.0),
    (65, 129, "fp16", "fp32", 1, True, True, "rms", -2.0),
    (300, 512, "fp32", "bf16", 4, True, True, "rms", 1.0),
    (41, 513, "bf16", "fp32", 2, True, False, "layer", 1.0),
    (1003, 1283, "fp16", "fp32", 1, True, True, "rms", 1.0),
    (517, 1000, "fp32", "fp32", 2, False, True, "layer", 0.7),
    (2050, 2048, "bf16", "bf16", 2, True, False, "layer", 1.0),
    (33, 4099, "fp32", "fp32", 1, False, False, "layer", 1.0),
    (130, 8191, "bf16", "fp16", 1, True, True, "layer", 1.0),
    (9, 8192, "fp32", "fp32", 3, False, True, "rms", 1.0),
    (400, 640, "bf16", "bf16", 300, True, True, "layer", 1.0),   # a group is one run
]


@pytest.mark.parametrize("M,C,dtype,pdtype,groups,one_plus,post,kind,alpha", CASES)
def test_against_float64(M, C, dtype, pdtype, groups, one_plus, post, kind, alpha):
    c = _case(M, C, TYPES[dtype], TYPES[pdtype], groups, one_plus, post, M + C)
    rpg = -(-M // groups)
    s, y, stats = S.residual_norm_forward(c["x"], c["h"], c["gate"], c["weight"], c["bias"], post_weight=c["post"], kind=kind,
                                          alpha=alpha, eps=1e-5, one_plus=one_plus, rows_per_group=rpg)
    _check_forward(c, kind, post, one_plus, rpg, alpha, 1e-5, s, y, stats)
    for ds in (c["ds"], None):
        got = S.residual_norm_backward(c["dy"], s, c["h"], stats, c["gate"], c["weight"], post_weight=c["post"], ds=ds, kind=kind,
                                       alpha=alpha, one_plus=one_plus, rows_per_group=rpg)
        _check_backward(c, s, stats, kind, post, one_plus, rpg, groups, alpha, got, TYPES[pdtype], False, ds)
    again = S.residual_norm_backward(c["dy"], s, c["h"], stats, c["gate"], c["weight"], post_weight=c["post"], kind=kind,
                                     alpha=alpha, one_plus=one_plus, rows_per_group=rpg)
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))
    assert S.residual_norm_backward(c["dy"], s, c["h"], stats, c["gate"], c["weight"], post_weight=c["post"], kind=kind,
                                    alpha=alpha, one_plus=one_plus, rows_per_group=rpg, param_grads=False)[2:] == (None,) * 4


@pytest.mark.parametrize("post", [False, True])
def test_without_parameters(post):
    c = _case(77, 321, torch.bfloat16, torch.float32, 1, False, False, 5)
    c.update(gate=None, weight=None, bias=None)
    s, y, stats = S.residual_norm_forward(c["x"], c["h"], post_norm=post)
    _check_forward(c, "layer", post, False, 77, 1.0, 1e-6, s, y, stats)
    got = S.residual_norm_backward(c["dy"], s, c["h"], stats, post_norm=post, grad_dtype=torch.float32)
    assert got[2].dtype == torch.float32 and got[2].shape == (321,)
    _check_backward(c, s, stats, "layer", post, False, 77, 1, 1.0, got, torch.float32, True, None)


def test_strides_in_place_and_vectors():
    """Rows apart, parameters that are slices of a modulation's output, the
    stream updated in place, odd alignment; what lies between rows stays."""
    M, C, dtype = 203, 515, torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(8)
    big = torch.randn(M, 3 * C + 1, device="cuda", generator=gen).to(dtype)
    x, h = big[:, 1:C + 1], big[:, C + 1:2 * C + 1]
    mod = torch.randn(2, 4 * C, device="cuda", generator=gen).to(dtype)
    p = [mod[:, i * C:(i + 1) * C] for i in range(4)]
    want = S.residual_norm_forward(x.contiguous(), h.contiguous(), *[t.contiguous() for t in p[:3]],
                                   post_weight=p[3].contiguous(), one_plus=True)
    before = big.clone()
    s, y, stats = S.residual_norm_forward(x, h, p[0], p[1], p[2], post_weight=p[3], one_plus=True, s=x, y=h)
    assert s.data_ptr() == x.data_ptr() and y.data_ptr() == h.data_ptr()
    for a, b in zip((s, y, stats), want):
        assert torch.equal(a, b)
    assert torch.equal(big[:, 0], before[:, 0]) and torch.equal(big[:, 2 * C + 1:], before[:, 2 * C + 1:])
    dy = torch.randn(M, C, device="cuda", generator=gen).to(dtype)
    ds = torch.randn(M, C, device="cuda", generator=gen).to(dtype)
    hh = before[:, C + 1:2 * C + 1].contiguous()
    args = dict(post_weight=p[3], one_plus=True)
    want = S.residual_norm_backward(dy, s.contiguous(), hh, stats, p[0], p[1], ds=ds, **args)
    h2 = hh.clone()
    got = S.residual_norm_backward(dy, s, h2, stats, p[0], p[1], ds=ds, dx=ds, dh=h2, **args)
    assert got[0] is ds and got[1] is h2
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_not_finite_rows_stay_alone():
    c = _case(40, 700, torch.bfloat16, torch.float32, 2, False, True, 3)
    rpg = 20
    run = lambda x, h: S.residual_norm_forward(x, h, c["gate"], c["weight"], c["bias"], post_weight=c["post"], kind="rms",   # noqa: E731
                                               rows_per_group=rpg)
    clean = run(c["x"], c["h"])
    x, h = c["x"].clone(), c["h"].clone()
    x[3, 5], h[30, 699] = float("nan"), float("inf")
    s, y, stats = run(x, h)
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[3] = rows[30] = False
    assert torch.equal(s[rows], clean[0][rows]) and torch.equal(y[rows], clean[1][rows])
    assert bool(y[3].isnan().all()) and bool(y[30].isnan().all())
    got = S.residual_norm_backward(c["dy"], s, h, stats, c["gate"], c["weight"], post_weight=c["post"], kind="rms", rows_per_group=rpg)
    want = S.residual_norm_backward(c["dy"], clean[0], c["h"], clean[2], c["gate"], c["weight"], post_weight=c["post"], kind="rms",
                                    rows_per_group=rpg)
    assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[1][rows], want[1][rows])


def test_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(3, 64, dtype=torch.float32, device="cuda")
    s, y, stats = S.residual_norm_forward(x, x, w, w, w)
    assert s.shape == (0, 64) and stats.shape == (2, 0)
    got = S.residual_norm_backward(x, s, x, stats, w, w)
    for g in got[2:5]:
        assert g.shape == (3, 64) and not bool(g.any())
    # groups behind the last row
    c = _case(10, 64, torch.bfloat16, torch.float32, 4, False, False, 3)
    s, y, stats = S.residual_norm_forward(c["x"], c["h"], c["gate"], c["weight"], c["bias"], rows_per_group=5)
    got = S.residual_norm_backward(c["dy"], s, c["h"], stats, c["gate"], c["weight"], rows_per_group=5)
    assert all(not bool(g[2:].any()) and bool(g[:2].any()) for g in got[2:5])


def test_stream_and_graph():
    c = _case(600, 1024, torch.bfloat16, torch.bfloat16, 2, True, True, 11)
    w = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")   # eager work between the replays

    def step():
        s, y, stats = S.residual_norm_forward(c["x"], c["h"], c["gate"], c["weight"], c["bias"], post_weight=c["post"], one_plus=True)
        return (s, y, stats) + S.residual_norm_backward(c["dy"], s, c["h"], stats, c["gate"], c["weight"], post_weight=c["post"],
                                                        ds=c["ds"], one_plus=True)
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s, y, stats = S.residual_norm_forward(c["x"], c["h"], c["gate"], c["weight"], c["bias"], post_weight=c["post"], one_plus=True,
                                          stream=side)
    got = S.residual_norm_backward(c["dy"], s, c["h"], stats, c["gate"], c["weight"], post_weight=c["post"], ds=c["ds"],
                                   one_plus=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((s, y, stats) + got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for t in out:
            t.zero_()
        w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        w.fill_(1)


def test_warns_outside_of_autograd():
    x = torch.randn(4, 64, device="cuda").requires_grad_()
    with pytest.warns(UserWarning, match="autograd"):
        S.residual_norm_forward(x, x)
    with pytest.raises(ValueError, match="h:"):
        S.residual_norm_forward(x.detach(), x.detach()[:2])
    with pytest.raises(ValueError, match="GPU"):
        S.residual_norm_forward(x.detach(), x.detach().cpu())

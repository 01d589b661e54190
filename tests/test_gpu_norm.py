"""svdq_layer_norm_forward and _backward against float64 (MI355X only).

Tolerances. u = 2^-24 is half a step of an fp32 operation. A sum over a row
takes at most D = 48 additions in a chain (16 in a lane, 6 over the wave, 16
waves, 2 for the scaling), so a mean of values v is off by D u mean|v|. The
bounds below add each operation's half step to first order; the last rounding
adds half a step of the output type."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import fp8_reference as R

pytestmark = pytest.mark.gpu

D, U = 48, R.F32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _inputs(M, C, dtype, pdtype, groups, seed, one_plus=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, C, device="cuda", generator=g) + 0.5
    if C > 3:
        x[:, C // 3] *= 30
    w = torch.randn(groups, C, device="cuda", generator=g) * 0.3 + (0.0 if one_plus else 1.0)
    b = torch.randn(groups, C, device="cuda", generator=g)
    dy = torch.randn(M, C, device="cuda", generator=g)
    return x.to(dtype), w.to(pdtype), b.to(pdtype), dy.to(dtype)


def _check_forward(x, w, b, eps, one_plus, rpg, y, mean, rstd, what):
    ref, rm, rr, xhat, gain = R.layer_norm(x, w, b, eps, one_plus, rpg)
    e_mean = (D + 2) * U * x.double().abs().mean(1)
    assert bool(((mean.double() - rm).abs() <= e_mean).all()), what
    e_rstd = (D / 2 + 6) * U + rr.square() * e_mean.square()
    assert bool(((rstd.double() / rr - 1).abs() <= e_rstd).all()), what
    e_xhat = rr[:, None] * e_mean[:, None] + xhat.abs() * (e_rstd[:, None] + 3 * U)
    shift = ref - xhat * gain
    bound = gain.abs() * e_xhat + 3 * U * (xhat * gain).abs() + U * shift.abs()
    bound = bound * (1 + R.half_step(x.dtype)) + R.half_step(x.dtype) * ref.abs() + 1e-12
    if x.dtype == torch.float16:
        bound = bound + 2.0 ** -25   # half of fp16's smallest step
    bad = (y.double() - ref).abs() > bound
    assert not bool(bad.any()), (what, int(bad.sum()), float(((y.double() - ref).abs() / bound).max()))


def _check_backward(dy, x, mean, rstd, w, one_plus, rpg, groups, dx, dw, db, what):
    dyd, xd = dy.double(), x.double()
    g = torch.arange(x.shape[0], device=x.device) // rpg
    gain = torch.ones_like(xd) if w is None else w.double()[g] + (1.0 if one_plus else 0.0)
    r = rstd.double()[:, None]
    xhat = (xd - mean.double()[:, None]) * r
    d = dyd * gain
    c1, c2 = d.mean(1, keepdim=True), (d * xhat).mean(1, keepdim=True)
    ref = r * (d - c1 - xhat * c2)
    bound = r * (3 * U * d.abs() + (D + 6) * U * d.abs().mean(1, keepdim=True)
                 + xhat.abs() * (D + 12) * U * (d * xhat).abs().mean(1, keepdim=True)
                 + 3 * U * (d.abs() + c1.abs() + (xhat * c2).abs()))
    bound = bound * (1 + R.half_step(x.dtype)) + R.half_step(x.dtype) * ref.abs() + 1e-12
    if x.dtype == torch.float16:
        bound = bound + 2.0 ** -25
    bad = (dx.double() - ref).abs() > bound
    assert not bool(bad.any()), (what, "dx", int(bad.sum()), float(((dx.double() - ref).abs() / bound).max()))
    for i in range(groups):
        rows = g == i
        n = int(rows.sum())
        # a lane's rows (a run's, shared by its teams), the teams (16, and 2 in a wave), the runs (8, then 32)
        runs = max(1, min(512 // max(1, -(-x.shape[0] // rpg)), -(-min(rpg, x.shape[0]) // 8)))
        chain = -(-n // runs) + 2 + 32 + 16 + 6
        for got, terms, name in ((dw, dyd * xhat, "dweight"), (db, dyd, "dbias")):
            want, mags = terms[rows].sum(0), terms[rows].abs().sum(0)
            lim = chain * U * mags * (1 + R.half_step(got.dtype)) + R.half_step(got.dtype) * want.abs() + 1e-12
            if got.dtype == torch.float16:
                lim = lim + 2.0 ** -25
            bad = (got[i].double() - want).abs() > lim
            assert not bool(bad.any()), (what, name, i, int(bad.sum()))


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 63), (2, 64), (7, 100), (4, 513), (33, 1024), (17, 1283), (9, 2048), (130, 3072),
          (6, 4097), (3, 8192), (2, 12289), (1, 16384), (2, 16383), (700, 33), (2051, 128)]


@pytest.mark.parametrize("dtype,pdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                          ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("M,C", SHAPES)
def test_norm_matches_float64(M, C, dtype, pdtype):
    groups, one_plus = (2 if M % 3 == 0 else 1), M % 2 == 0
    x, w, b, dy = _inputs(M, C, TYPES[dtype], TYPES[pdtype], groups, M * 7 + C, one_plus)
    rpg = -(-M // groups)
    y, mean, rstd = S.layer_norm_forward(x, w, b, eps=1e-5, one_plus=one_plus, rows_per_group=rpg)
    _check_forward(x, w, b, 1e-5, one_plus, rpg, y, mean, rstd, (M, C, dtype))
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w, one_plus=one_plus, rows_per_group=rpg)
    assert dw.shape == (groups, C) and dw.dtype == TYPES[pdtype]
    _check_backward(dy, x, mean, rstd, w, one_plus, rpg, groups, dx, dw, db, (M, C, dtype))


@pytest.mark.parametrize("M,C,rpg,groups", [(1000, 264, 100, 10), (1000, 264, 333, 5), (64, 40, 1, 64),
                                            (40, 40, 1, 700), (9000, 72, 9000, 1), (9001, 72, 4000, 3)])
def test_norm_groups(M, C, rpg, groups):
    """Groups of any length; groups without rows get zero gradients."""
    x, w, b, dy = _inputs(M, C, torch.float32, torch.float32, groups, C)
    y, mean, rstd = S.layer_norm_forward(x, w, b, rows_per_group=rpg)
    _check_forward(x, w, b, 1e-6, False, rpg, y, mean, rstd, (M, rpg))
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=rpg)
    _check_backward(dy, x, mean, rstd, w, False, rpg, groups, dx, dw, db, (M, rpg))
    dx2, dw2, db2 = S.layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=rpg)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_norm_without_parameters_and_partial_outputs():
    x, w, b, dy = _inputs(37, 200, torch.bfloat16, torch.bfloat16, 1, 5)
    y, mean, rstd = S.layer_norm_forward(x)
    _check_forward(x, None, None, 1e-6, False, 37, y, mean, rstd, "plain")
    y1, *_ = S.layer_norm_forward(x, bias=b)
    _check_forward(x, None, b, 1e-6, False, 37, y1, mean, rstd, "bias only")
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd)
    assert dw.shape == (200,) and dw.dtype == torch.float32
    _check_backward(dy, x, mean, rstd, None, False, 37, 1, dx, dw[None], db[None], "plain")
    dx2, none, none2 = S.layer_norm_backward(dy, x, mean, rstd, param_grads=False)
    assert none is None and none2 is None and torch.equal(dx, dx2)
    flat = S.layer_norm_backward(dy, x, mean, rstd, w[0], grad_dtype=torch.float32)
    assert flat[1].shape == (200,) and flat[1].dtype == torch.float32


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_strides_and_in_place(dtype):
    """Row strides of x, y, dy, dx and of the parameters; rows around the
    written ones stay; y may be x and dx may be dy."""
    M, C = 50, 77
    wide, mod, b, wide_dy = (torch.randn(s, device="cuda").to(TYPES[dtype]) for s in
                             ((M, 100), (2, 6 * C), (2, 6 * C), (M, 91)))
    x, w, sh, dy = wide[:, 11:11 + C], mod[:, C:2 * C], b[:, 3 * C:4 * C], wide_dy[:, 5:5 + C]
    out = torch.full((M + 2, 120), 7.0, dtype=TYPES[dtype], device="cuda")
    y, mean, rstd = S.layer_norm_forward(x, w, sh, one_plus=True, rows_per_group=25, y=out[1:M + 1, 9:9 + C])
    _check_forward(x, w, sh, 1e-6, True, 25, y, mean, rstd, "strided")
    assert bool((out[0] == 7).all() and (out[M + 1] == 7).all() and (out[:, :9] == 7).all() and (out[:, 9 + C:] == 7).all())
    dout = torch.full((M + 2, 120), 7.0, dtype=TYPES[dtype], device="cuda")
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w, one_plus=True, rows_per_group=25, dx=dout[1:M + 1, 3:3 + C])
    _check_backward(dy, x, mean, rstd, w, True, 25, 2, dx, dw, db, "strided")
    assert bool((dout[0] == 7).all() and (dout[M + 1] == 7).all() and (dout[:, :3] == 7).all() and (dout[:, 3 + C:] == 7).all())
    keep_x, keep_dy = x.clone(), dy.clone()
    dx2, _, _ = S.layer_norm_backward(dy, x, mean, rstd, w, one_plus=True, rows_per_group=25, dx=dy)
    assert torch.equal(dx2, dx)
    y2, _, _ = S.layer_norm_forward(x, w, sh, one_plus=True, rows_per_group=25, y=x)
    assert torch.equal(y2, y) and not torch.equal(keep_x, x) and not torch.equal(keep_dy, dy)


def test_norm_infinities_and_nan_stay_in_their_row():
    x, w, b, dy = _inputs(12, 300, torch.bfloat16, torch.bfloat16, 1, 8)
    x[3, 7], x[5, 0], x[9, 299] = float("inf"), float("nan"), float("-inf")
    y, mean, rstd = S.layer_norm_forward(x, w, b)
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w)
    bad = torch.zeros(12, dtype=torch.bool, device="cuda")
    bad[[3, 5, 9]] = True
    assert bool(y[bad].isnan().all()) and bool(y[~bad].isfinite().all())
    assert bool(dx[bad].isnan().all()) and bool(dx[~bad].isfinite().all())
    assert bool(dw.isnan().all()) and bool(db.isfinite().all())


def test_norm_constant_rows_and_large_offset():
    """A constant row gives the bias (eps > 0); a mean far above the deviation
    keeps its digits (two passes)."""
    b = torch.randn(100, device="cuda")
    y, mean, rstd = S.layer_norm_forward(torch.full((3, 100), 2.5, device="cuda"), None, b)
    assert torch.equal(y, b.expand(3, 100)) and bool((mean == 2.5).all())
    x = torch.randn(4, 1000, device="cuda") + 4096.0
    y, mean, rstd = S.layer_norm_forward(x)
    _check_forward(x, None, None, 1e-6, False, 4, y, mean, rstd, "offset")


def test_norm_gradient_against_differences():
    """dx and dweight against central differences of the float64 forward."""
    M, C, h = 2, 24, 1e-4
    x, w, b, dy = _inputs(M, C, torch.float32, torch.float32, 1, 3)
    y, mean, rstd = S.layer_norm_forward(x, w, b)
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w)

    def loss(xx, ww):
        off = xx - xx.mean(1, keepdim=True)
        return (dy.double() * (off / torch.sqrt(off.square().mean(1, keepdim=True) + 1e-6) * ww)).sum()

    xd, wd = x.double(), w.double()
    for i in range(M):
        for j in range(C):
            e = torch.zeros_like(xd)
            e[i, j] = h
            diff = (loss(xd + e, wd) - loss(xd - e, wd)) / (2 * h)
            # h^2 times a third derivative of order 10, and the fp32 bound
            assert abs(float(dx[i, j]) - float(diff)) <= 1e-6 + 1e-5 * abs(float(diff))
    for j in range(C):
        e = torch.zeros_like(wd)
        e[0, j] = h
        diff = (loss(xd, wd + e) - loss(xd, wd - e)) / (2 * h)
        assert abs(float(dw[0, j]) - float(diff)) <= 1e-5 + 1e-5 * abs(float(diff))


def test_norm_empty():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = S.layer_norm_forward(x, torch.ones(64, device="cuda"))
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = S.layer_norm_backward(x, x, mean, rstd, torch.ones(2, 64, device="cuda"), rows_per_group=3)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


def test_norm_on_another_stream_and_in_a_graph():
    x, w, b, dy = _inputs(600, 640, torch.bfloat16, torch.bfloat16, 2, 21)
    y0, mean0, rstd0 = S.layer_norm_forward(x, w, b, rows_per_group=300)
    g0 = S.layer_norm_backward(dy, x, mean0, rstd0, w, rows_per_group=300)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y1, mean1, rstd1 = S.layer_norm_forward(x, w, b, rows_per_group=300, stream=side)
    g1 = S.layer_norm_backward(dy, x, mean1, rstd1, w, rows_per_group=300, stream=side)
    side.synchronize()
    assert torch.equal(y0, y1) and all(torch.equal(a, c) for a, c in zip(g0, g1))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        yg, mg, rg = S.layer_norm_forward(x, w, b, rows_per_group=300)
        gg = S.layer_norm_backward(dy, x, mg, rg, w, rows_per_group=300)
    for k in range(3):
        x.copy_(torch.randn(600, 640, device="cuda").to(torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        y, mean, rstd = S.layer_norm_forward(x, w, b, rows_per_group=300)
        e = S.layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=300)
        assert torch.equal(y, yg) and all(torch.equal(a, c) for a, c in zip(e, gg)), k


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,C,rpg", [(513, 250, 100), (300, 129, 7), (1000, 64, 333), (77, 16, 1), (50, 3, 20), (9, 2, 1 << 40),
                                     (2051, 65, 1000), (20, 5000, 9), (12, 12288, 12), (5, 15001, 3), (260, 6000, 130),
                                     (40, 9000, 40), (64, 1537, 64)])
def test_norm_teams(M, C, rpg, dtype):
    """Rows that share a wave (also of different groups), rows shorter than a
    vector, rows of a wave and of many."""
    groups = (M - 1) // rpg + 1
    x, w, b, dy = _inputs(M, C, TYPES[dtype], torch.float32, groups, M + C, True)
    y, mean, rstd = S.layer_norm_forward(x, w, b, one_plus=True, rows_per_group=rpg)
    _check_forward(x, w, b, 1e-6, True, rpg, y, mean, rstd, (M, C, rpg))
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w, one_plus=True, rows_per_group=rpg)
    _check_backward(dy, x, mean, rstd, w, True, rpg, groups, dx, dw, db, (M, C, rpg))
    again = S.layer_norm_backward(dy, x, mean, rstd, w, one_plus=True, rows_per_group=rpg)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


def test_norm_refuses_overlapping_rows():
    """Expanded tensors (rows or groups a stride of 0 apart) and rows closer
    than their length are errors, not other memory."""
    x, w, b, dy = _inputs(6, 40, torch.bfloat16, torch.bfloat16, 2, 1)
    y, mean, rstd = S.layer_norm_forward(x, w, b)
    one = x[:1].expand(6, 40)
    with pytest.raises(ValueError):
        S.layer_norm_forward(one)
    with pytest.raises(ValueError):
        S.layer_norm_forward(x, y=one)
    with pytest.raises(ValueError):
        S.layer_norm_forward(x, w[:1].expand(2, 40))
    with pytest.raises(ValueError):
        S.layer_norm_forward(x, w, b[:1].expand(2, 40))
    with pytest.raises(ValueError):
        S.layer_norm_forward(x.reshape(-1).as_strided((6, 40), (39, 1)))
    with pytest.raises(ValueError):
        S.layer_norm_forward(x.t())
    with pytest.raises(ValueError):
        S.layer_norm_backward(one, x, mean, rstd, w)
    with pytest.raises(ValueError):
        S.layer_norm_backward(dy, x, mean[:1].expand(6), rstd, w)


@pytest.mark.parametrize("C", [5, 40, 100, 250])
def test_norm_infinities_and_nan_in_rows_that_share_a_wave(C):
    x, w, b, dy = _inputs(40, C, torch.bfloat16, torch.bfloat16, 1, 8)
    x[3, C // 2], x[17, 0], x[38, C - 1] = float("inf"), float("nan"), float("-inf")
    y, mean, rstd = S.layer_norm_forward(x, w, b)
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[3, 17, 38]] = True
    assert bool(y[bad].isnan().all()) and bool(y[~bad].isfinite().all())
    assert bool(dx[bad].isnan().all()) and bool(dx[~bad].isfinite().all())
    assert bool(db.isfinite().all())

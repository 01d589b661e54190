"""FP8 products over every tile of the persistent kernel, several tiles a
workgroup, and inputs large enough to be read past the caches, against float64
(MI355X only). The shapes are fp8_cases.py's."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import fp8_cases as C
from tests import fp8_reference as R
from tests.test_gpu_fp8 import _bf16, _close, _codes, _layer, _weight
from tests.test_gpu_norm import TYPES, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tile,blocks,M,K,N", C.FORWARD)
def test_forward(tile, blocks, M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    x = _bf16(g, M, K)
    _, dev = _layer(g, K, N, transposed=False)
    room = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = S.fp8_forward(K, N, dev, x, y=room[1:M + 1])
    a, w = R.q8(x.double())[0], _weight(dev, K, N)
    bias = dev["bias"].double()
    _close(y, a @ w.t().contiguous() + bias, R.product_bound(a, w, bias), (M, K, N))
    assert bool((room[0] == 7).all()) and bool((room[M + 1] == 7).all())
    assert torch.equal(y, S.fp8_forward(K, N, dev, x))


@pytest.mark.parametrize("tile,blocks,M,K,N", C.BACKWARD)
def test_weight_gradient(tile, blocks, M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    x, dy = _bf16(g, M, K), _bf16(g, M, N, scale=1e-3)
    _, dev = _layer(g, K, N, bias=False)
    dx, dw, db = S.fp8_backward(K, N, dev, x, dy)
    ty, tx = R.q8(dy.double(), 0)[0].t().contiguous(), R.q8(x.double(), 0)[0].t().contiguous()
    _close(dw, ty @ tx.t().contiguous(), R.product_bound(ty, tx), ("dw", M, K, N))
    del ty, tx
    a, w = R.q8(dy.double())[0], _weight(dev, K, N)
    _close(dx, a @ w, R.product_bound(a, w.t().contiguous()), ("dx", M, K, N))
    want, mags = dy.double().sum(0), dy.double().abs().sum(0)
    _close(db, want, (2 + 16 + 1 + M / 128 + 1) * R.F32 * mags + R.half_step(torch.bfloat16) * want.abs() * 1.001,
           ("db", M, K, N), many=False)
    again = S.fp8_backward(K, N, dev, x, dy)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("M,K", C.QUANTIZED)
def test_quantizer_bits_of_large_inputs(M, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = _bf16(g, M, K)
    q, s = S.fp8_quantize(x)
    want, e = R.q8(x.double())
    byte = torch.stack([s[b // 4, :, b % 4] for b in range(-(-K // 128))], 1).double()
    assert torch.equal(byte, e + 127)
    assert torch.equal(_codes(q)[:, :K], want * torch.exp2(-e).repeat_interleave(128, 1)[:, :K])


def _chain(M, C, rows_per_group, groups, elem_bytes):
    """The additions in a row that a value of a parameter gradient goes through
    at most, from the plan of the kernels: a row belongs to a team of lanes
    that hold 16 elements each at most (a quarter or half wave, or whole
    waves); a workgroup of up to 16 waves (12 with more than 12 elements a
    lane) has as many teams as fit and have rows, and takes one run of a
    group's rows, about 256 runs in all of at least four rows, or one where
    its teams have two rows each at most. A lane adds its rows, the teams of a
    wave are added pairwise, the waves' in order, then the runs: 32 chains of
    every 32nd run, and the 32."""
    vec = 16 // elem_bytes
    n = -(-C // vec)
    if n <= 32:
        nv, waves, sub = 1, 1, 4 if n <= 16 else 2
    else:
        fits = [(nv * w, -nv, nv, w) for nv in range(1, 16 // vec + 1) for w in [-(-n // (64 * nv))]
                if w <= 16 and -(-n // (64 * w)) == nv]
        _, _, nv, waves = min(fits)
        sub = 1
    most = 12 if nv * vec > 12 else 16
    teams = max(1, most // waves) * sub
    rows = min(rows_per_group, M)
    runs = min(256 // -(-M // rows_per_group), -(-rows // 4))
    if runs < 1 or groups > 256 or rows <= 2 * teams:
        runs = 1
    of_run = -(-rows // runs)
    here = min(teams // sub, -(-of_run // sub)) * sub
    joined = -(-runs // 32) + 31 if runs > 1 else 0
    return -(-of_run // here) + {1: 0, 2: 1, 4: 2}[sub] + here // sub - 1 + joined


@pytest.mark.parametrize("M,C_,dtype,groups", [(M, c, t, 1 + i) for i, (M, c, t) in enumerate(C.NORM_GRADIENTS)]
                         + [(700, 33, "bf16", 1), (2051, 128, "fp32", 2), (9001, 72, "fp32", 3), (513, 250, "fp16", 6),
                            (3000, 1283, "bf16", 1), (260, 6000, "fp32", 2)])
def test_norm_gradients_within_the_present_plans_bound(M, C_, dtype, groups):
    x, w, b, dy = _inputs(M, C_, TYPES[dtype], torch.float32, groups, M)
    rpg = -(-M // groups)
    _, mean, rstd = S.layer_norm_forward(x, w, b, rows_per_group=rpg)
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=rpg)
    xhat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for i in range(groups):
        rows = slice(i * rpg, min((i + 1) * rpg, M))
        d, t = dy[rows].double(), dy[rows].double() * xhat[rows]
        chain = _chain(M, C_, rpg, groups, x.element_size())
        # xhat has two roundings; its product with dy is rounded with the addition
        for got, terms, extra in ((dw, t, 2), (db, d, 0)):
            want, mags = terms.sum(0), terms.abs().sum(0)
            assert bool(((got[i].double() - want).abs() <= 1.001 * (chain + extra) * R.F32 * mags).all()), (M, C_, i, extra)
        g = w[i].double()
        dd = d * g
        c1, c2 = dd.mean(1, keepdim=True), (dd * xhat[rows]).mean(1, keepdim=True)
        r = rstd[rows].double()[:, None]
        ref = r * (dd - c1 - xhat[rows] * c2)
        # as in test_gpu_norm.py: 48 additions of a row's sums
        bound = r * R.F32 * (3 * dd.abs() + 54 * dd.abs().mean(1, keepdim=True)
                             + xhat[rows].abs() * 60 * (dd * xhat[rows]).abs().mean(1, keepdim=True)
                             + 3 * (dd.abs() + c1.abs() + (xhat[rows] * c2).abs()))
        half = R.half_step(x.dtype)
        bound = bound * (1 + half) + half * ref.abs() + (2.0 ** -25 if dtype == "fp16" else 1e-12)
        assert bool(((dx[rows].double() - ref).abs() <= bound).all()), (M, C_, i)
    again = S.layer_norm_backward(dy, x, mean, rstd, w, rows_per_group=rpg)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))

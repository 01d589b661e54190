"""Layer norm and FP8 linear where offsets pass 2^31 and 2^32 (MI355X only):
the last rows and channels against float64, or against a call on them alone."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import fp8_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free GPU memory")
    yield
    torch.cuda.empty_cache()


def _bf16(g, *shape, scale=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g).mul_(scale)


def _ends(n, k=70):
    """The first and the last k of n."""
    return torch.cat([torch.arange(k), torch.arange(n - k, n)]).cuda()


def test_norm_of_many_wide_rows():
    """70000 x 16384 fp32, 4.6 GB each of x, y, dy and dx: a row's results are
    those of its row alone."""
    M, C = 70000, 16384
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.empty(M, C, device="cuda").normal_(generator=g) for _ in range(2))
    y, mean, rstd = S.layer_norm_forward(x)
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd)
    for rows in (slice(0, 9), slice(32765, 32772), slice(65533, 65540), slice(M - 9, M)):
        few, few_dy = x[rows].contiguous(), dy[rows].contiguous()
        y1, m1, r1 = S.layer_norm_forward(few)
        dx1 = S.layer_norm_backward(few_dy, few, m1, r1, param_grads=False)[0]
        assert torch.equal(y[rows], y1) and torch.equal(mean[rows], m1) and torch.equal(rstd[rows], r1)
        assert torch.equal(dx[rows], dx1)
    want = torch.zeros(C, dtype=torch.float64, device="cuda")
    mags = torch.zeros_like(want)
    for at in range(0, M, 7000):
        part = dy[at:at + 7000].double()
        want += part.sum(0)
        mags += part.abs().sum(0)
    # a run's 274 rows, one team a workgroup, then 8 and 32 runs: fewer than 320 additions
    assert bool(((db.double() - want).abs() <= 320 * R.F32 * mags).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rows_far_apart(dtype):
    """Rows 2^31 + 24 elements apart."""
    M, C, ld = 3, 1000, (1 << 31) + 24
    g = torch.Generator(device="cuda").manual_seed(2)
    room = torch.zeros((M - 1) * ld + C + 8, dtype=dtype, device="cuda")
    far = room.as_strided((M, C), (ld, 1), 5)
    x, dy = torch.randn(M, C, device="cuda", generator=g).to(dtype), torch.randn(M, C, device="cuda", generator=g).to(dtype)
    far.copy_(x)
    y, mean, rstd = S.layer_norm_forward(x)
    dx, dw, db = S.layer_norm_backward(dy, x, mean, rstd)
    got = S.layer_norm_backward(dy, far, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, (dx, dw, db)))
    S.layer_norm_forward(far, y=far)
    assert torch.equal(far, y)
    S.layer_norm_backward(dy, x, mean, rstd, dx=far)
    assert torch.equal(far, dx)
    far.zero_()
    assert int(room.count_nonzero()) == 0


@pytest.mark.parametrize("M", [3, 40])
def test_the_largest_layer(M):
    """65536 -> 65536 channels: 4.3 GB of codes, 8.6 GB of weight gradient."""
    K = N = 65536
    g = torch.Generator(device="cuda").manual_seed(M)
    w = _bf16(g, N, K, scale=1 / 256)
    dev = S.fp8_pack(w)
    x, dy = _bf16(g, M, K), _bf16(g, M, N, scale=1e-3)
    rows, cols = _ends(N), _ends(K)
    # the packed layer against its definition, at the corners
    for n0 in (0, N - 128):
        q, e = R.q8_blocks(w[n0:n0 + 128].double())
        assert torch.equal(dev["s"][n0 // 128, :512].double(), e[0] + 127)
        assert torch.equal(dev["q"][n0:n0 + 128].view(torch.float8_e4m3fn).double(),
                           q * torch.exp2(-e).repeat_interleave(128, 1))
    assert torch.equal(dev["qt"][cols], dev["q"][:, cols].t()) and torch.equal(dev["st"][:, :512], dev["s"][:, :512].t())
    del w

    def weight(codes, scales, at):
        """Rows `at` of codes [.][65536] with scales [512][512], as float64."""
        e = scales[(at // 128), :512].double() - 127
        return codes[at].view(torch.float8_e4m3fn).double() * torch.exp2(e).repeat_interleave(128, 1)

    def close(got, a, b, what):
        want, bound = a @ b.t().contiguous(), R.product_bound(a, b)
        assert bool(((got.double() - want).abs() <= bound).all()), what

    close(S.fp8_forward(K, N, dev, x)[:, rows], R.q8(x.double())[0], weight(dev["q"], dev["s"], rows), "y")
    dx, dw, db = S.fp8_backward(K, N, dev, x, dy)
    close(dx[:, cols], R.q8(dy.double())[0], weight(dev["qt"], dev["st"], cols), "dx")
    ty, tx = R.q8(dy.double(), 0)[0].t().contiguous(), R.q8(x.double(), 0)[0].t().contiguous()
    close(dw[rows], ty[rows].contiguous(), tx, "dw")
    close(dw[:, cols], ty, tx[cols].contiguous(), "dw")
    want = dy.double().sum(0)   # fewer than 50 additions, one rounding
    assert bool(((db.double() - want).abs() <= 50 * R.F32 * dy.double().abs().sum(0) + 2.0 ** -8 * 1.001 * want.abs()).all())


def test_a_million_tokens():
    """2^20 tokens of 4112 channels: 8.6 GB of activations, 4.3 GB of
    transposed codes."""
    M, K, N = 1 << 20, 4112, 48
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = _bf16(g, M, K), _bf16(g, M, N, scale=1e-3)
    dev = S.fp8_pack(torch.randn(N, K, device="cuda", generator=g) / 64)
    rows = _ends(M)
    e = (dev["s"].double()[:, :33] - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    w = dev["q"].view(torch.float8_e4m3fn).double() * torch.exp2(e)
    for norm in (False, True):
        y = S.fp8_norm_forward(K, N, dev, x) if norm else S.fp8_forward(K, N, dev, x)
        part = x[rows].contiguous()
        a = R.q8((S.layer_norm_forward(part)[0] if norm else part).double())[0]
        assert bool(((y[rows].double() - a @ w.t().contiguous()).abs() <= R.product_bound(a, w)).all()), norm
    dx, dw, _ = S.fp8_backward(K, N, dev, x, dy)
    a = R.q8(dy[rows].double())[0]
    wt = w.t().contiguous()
    assert bool(((dx[rows].double() - a @ w).abs() <= R.product_bound(a, wt)).all())
    cols = _ends(K, 8)
    ty, tx = R.q8(dy.double(), 0)[0].t().contiguous(), R.q8(x[:, cols].double(), 0)[0].t().contiguous()
    want, bound = ty @ tx.t().contiguous(), R.product_bound(ty, tx)
    assert bool(((dw[:, cols].double() - want).abs() <= bound).all())


def test_the_most_tokens():
    """2^24 tokens of the forward."""
    M, K, N = 1 << 24, 16, 16
    g = torch.Generator(device="cuda").manual_seed(6)
    x = _bf16(g, M, K)
    dev = S.fp8_pack(torch.randn(N, K, device="cuda", generator=g))
    w = dev["q"].view(torch.float8_e4m3fn).double() * 2.0 ** (float(dev["s"][0, 0]) - 127)
    y = S.fp8_forward(K, N, dev, x)
    for at in range(0, M, 1 << 21):
        a = R.q8(x[at:at + (1 << 21)].double())[0]
        assert bool(((y[at:at + (1 << 21)].double() - a @ w.t().contiguous()).abs() <= R.product_bound(a, w)).all()), at

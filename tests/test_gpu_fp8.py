"""The FP8 linear (svdq_fp8_*) against float64 on the same inputs (MI355X
only): codes and scales bit for bit, products within the bound that
fp8_reference.product_bound derives."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import fp8_reference as R

pytestmark = pytest.mark.gpu


def _bf16(g, *shape, scale=1.0, outliers=True):
    v = torch.randn(*shape, device="cuda", generator=g) * scale
    if outliers and shape[-1] > 20:
        v[..., shape[-1] // 7] *= 50
    return v.to(torch.bfloat16)


def _layer(g, K, N, bias=True, transposed=True):
    w = torch.randn(N, K, device="cuda", generator=g) / K ** 0.5
    b = torch.randn(N, device="cuda", generator=g).to(torch.bfloat16) if bias else None
    return w, S.fp8_pack(w, b, transposed=transposed)


def _codes(q):
    return q.view(torch.float8_e4m3fn).double()


def _weight(dev, K, N):
    """The weight that the packed codes and scales stand for."""
    e = dev["s"].double()[:, :-(-K // 128)] - 127
    e = e.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return _codes(dev["q"]) * torch.exp2(e)


def _close(got, want, bound, what, many=True):
    """Every value within its bound and, with many values, together within
    bf16's rounding (an error spread over a step has 2^-8 / sqrt(3) = 2.3e-3 of
    the value; a single value, or one channel that holds nearly the whole norm
    as in db below, may be off by the half step 2^-8 = 3.9e-3)."""
    assert float((got.double() - want).norm()) <= (2.5e-3 if many else 2.0 ** -8 * 1.001) * float(want.norm()), what
    err = (got.double() - want).abs()
    bad = err > bound
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / bound.clamp(min=1e-300)).max()))


@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (5, 144), (17, 1024), (9, 2064), (130, 3072), (2, 65536)])
def test_quantizer_bits(M, K):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = _bf16(g, M, K)
    x[0, :K // 2] = 0                      # zero blocks and halves
    if M > 2:
        x[1] = x[1] * 2.0 ** 100           # large
        x[2] = x[2] * 2.0 ** -130          # subnormal bf16
    q, s = S.fp8_quantize(x)
    want, e = R.q8(x.double())
    nb = -(-K // 128)
    byte = torch.stack([s[b // 4, :, b % 4] for b in range(nb)], 1).double()
    assert torch.equal(byte, e + 127)
    scale = torch.exp2(e).repeat_interleave(128, 1)[:, :K]
    assert torch.equal(_codes(q)[:, :K], want / scale)
    assert bool((q[:, K:] == 0).all())


def test_quantizer_border_of_the_scale():
    """max|v| = 448 2^e keeps e, the next bf16 value takes e + 1; ties of the
    codes go to even."""
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[1, 0] = 448.0, 450.0
    x[2, :4] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10], device="cuda")   # 16|18, 18|20, 0|2^-9
    x[3, :3] = torch.tensor([-448.0, -17.0, 3 * 2.0 ** -10], device="cuda")
    q, s = S.fp8_quantize(x)
    assert s[0, :, 0].tolist() == [127, 128, 127, 127]
    c = _codes(q)
    assert c[2, :4].tolist() == [448.0, 16.0, 20.0, 0.0] and c[3, :3].tolist() == [-448.0, -16.0, 2.0 ** -8]


def test_quantizer_infinities_and_nan():
    x = torch.ones(3, 256, dtype=torch.bfloat16, device="cuda")
    x[0, 3], x[1, 200], x[2, 5] = float("inf"), float("nan"), float("-inf")
    q, _ = S.fp8_quantize(x)
    nan = _codes(q).isnan()
    assert nan.nonzero().tolist() == [[0, 3], [1, 200], [2, 5]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K,N", [(16, 16), (128, 128), (144, 272), (2064, 1552), (400, 528)])
def test_pack_bits(K, N, dtype):
    g = torch.Generator(device="cuda").manual_seed(K)
    w = (torch.randn(N, K, device="cuda", generator=g) / K ** 0.5).to(dtype)
    w[:16, :16] *= 20
    dev = S.fp8_pack(w)
    want, e = R.q8_blocks(w.double())
    rk, rn = -(-K // 128), -(-N // 128)
    assert torch.equal(dev["s"][:, :rk].double(), e + 127) and bool((dev["s"][:, rk:] == 0).all())
    assert torch.equal(dev["st"][:, :rn].double(), e.t() + 127) and bool((dev["st"][:, rn:] == 0).all())
    assert torch.equal(_weight(dev, K, N), want)
    assert torch.equal(dev["qt"], dev["q"].t().contiguous())
    again = S.fp8_pack(w * 3, out=dev)
    assert again is dev and torch.equal(_weight(dev, K, N), R.q8_blocks((w * 3).double())[0])


FORWARD = [(1, 16, 16), (1, 3072, 1040), (2, 144, 48), (7, 1040, 272), (15, 128, 128), (16, 2064, 400), (17, 400, 144),
           (31, 1552, 512), (33, 512, 1552), (64, 2176, 272), (65, 256, 256), (100, 144, 1040), (128, 128, 128),
           (129, 272, 144), (200, 640, 384), (257, 1040, 528), (300, 16, 16), (1003, 2064, 1552), (2, 65536, 32),
           (70, 32, 65536), (2100, 528, 4112)]


@pytest.mark.parametrize("M,K,N", FORWARD)
def test_forward(M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    x = _bf16(g, M, K)
    _, dev = _layer(g, K, N, bias=M % 2 == 1, transposed=False)
    ws = torch.full((max(1, S.fp8_workspace_bytes(K, N, M)),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    y = S.fp8_forward(K, N, dev, x, y=out[1:M + 1], workspace=ws)
    a, w = R.q8(x.double())[0], _weight(dev, K, N)
    bias = dev["bias"].double() if dev["bias"] is not None else 0.0
    _close(y, a @ w.t().contiguous() + bias, R.product_bound(a, w, bias), (M, K, N))
    assert bool((out[0] == 7).all()) and bool((out[M + 1] == 7).all())
    assert torch.equal(y, S.fp8_forward(K, N, dev, x))


@pytest.mark.parametrize("M", [5, 40, 300])
def test_forward_nan_stays_in_its_row_and_channel(M):
    """Infinities and NaN of a token reach its row only, a NaN code of the
    weight its channel only, also where the row after it continues in memory."""
    g = torch.Generator(device="cuda").manual_seed(M)
    K, N = 144, 160
    x = _bf16(g, M, K)
    x[1, 3], x[M - 1, K - 1] = float("inf"), float("nan")
    _, dev = _layer(g, K, N)
    dev["q"][7, 0] = 0x7F
    y = S.fp8_forward(K, N, dev, x)
    nan = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    nan[1], nan[M - 1], nan[:, 7] = True, True, True
    assert torch.equal(y.isnan(), nan)


@pytest.mark.parametrize("fmt_rows", [(1, 16), (16, 17), (64, 65)])
def test_row_does_not_depend_on_the_batch_within_a_path(fmt_rows):
    """A token's output is the same bits alone and in a batch on the few-token
    path, and within the bound across the paths."""
    g = torch.Generator(device="cuda").manual_seed(3)
    K, N = 1040, 272
    few, more = fmt_rows
    x = _bf16(g, more, K)
    _, dev = _layer(g, K, N)
    big, small = S.fp8_forward(K, N, dev, x), S.fp8_forward(K, N, dev, x[:few].contiguous())
    if more <= 16:
        assert torch.equal(big[:few], small)
    a, w = R.q8(x.double())[0], _weight(dev, K, N)
    bound = R.product_bound(a, w, dev["bias"].double())
    assert bool(((big[:few].double() - small.double()).abs() <= 2 * bound[:few]).all())


def test_forward_is_exact_on_whole_numbers():
    """Small whole numbers lose nothing to the quantizer and to fp32 sums."""
    g = torch.Generator(device="cuda").manual_seed(5)
    for M, K, N in [(3, 272, 48), (50, 144, 144), (260, 400, 272)]:
        x = torch.randint(-8, 9, (M, K), device="cuda", generator=g).to(torch.bfloat16)
        w = torch.randint(-4, 5, (N, K), device="cuda", generator=g).float()
        y = S.fp8_forward(K, N, S.fp8_pack(w), x)
        assert torch.equal(y, (x.double() @ w.double().t().contiguous()).to(torch.bfloat16))


@pytest.mark.parametrize("M,K,N,groups", [(1, 128, 64, 1), (5, 144, 272, 2), (40, 3072, 144, 2), (300, 1040, 528, 3),
                                          (64, 400, 48, 64), (20, 16, 16, 1), (9, 8208, 32, 1)])
def test_norm_forward_is_the_composition(M, K, N, groups):
    g = torch.Generator(device="cuda").manual_seed(M * K)
    x = _bf16(g, M, K)
    mod = _bf16(g, groups, 6 * K, scale=0.3, outliers=False)
    scale, shift = mod[:, K:2 * K], mod[:, :K]
    _, dev = _layer(g, K, N)
    rpg = -(-M // groups)
    ws = torch.full((S.fp8_norm_workspace_bytes(K, N, M),), 0xFF, dtype=torch.uint8, device="cuda")
    y, mean, rstd = S.fp8_norm_forward(K, N, dev, x, scale, shift, one_plus=True, rows_per_group=rpg, workspace=ws,
                                       stats=True)
    h, m2, r2 = S.layer_norm_forward(x, scale, shift, one_plus=True, rows_per_group=rpg)
    assert torch.equal(mean, m2) and torch.equal(rstd, r2)
    if M > 16:
        assert torch.equal(y, S.fp8_forward(K, N, dev, h))
    q, _ = S.fp8_quantize(h)
    assert torch.equal(ws[:q.numel()].view(q.shape), q)
    a, w = R.q8(h.double())[0], _weight(dev, K, N)
    bias = dev["bias"].double()
    _close(y, a @ w.t().contiguous() + bias, R.product_bound(a, w, bias), (M, K, N))


BACKWARD = [(1, 16, 16), (1, 144, 272), (7, 128, 128), (64, 400, 144), (65, 272, 400), (127, 144, 160), (128, 256, 256),
            (129, 528, 272), (300, 1040, 400), (777, 1552, 2064), (640, 144, 4112), (2500, 272, 272)]


@pytest.mark.parametrize("M,K,N", BACKWARD)
def test_backward(M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    x, dy = _bf16(g, M, K), _bf16(g, M, N, scale=1e-3)
    _, dev = _layer(g, K, N)
    ws = torch.full((S.fp8_backward_workspace_bytes(K, N, M),), 0xFF, dtype=torch.uint8, device="cuda")
    dx, dw, db = S.fp8_backward(K, N, dev, x, dy, workspace=ws)
    w = _weight(dev, K, N)
    a = R.q8(dy.double())[0]
    _close(dx, a @ w, R.product_bound(a, w.t().contiguous()), ("dx", M, K, N))
    ty, tx = R.q8(dy.double(), 0)[0].t().contiguous(), R.q8(x.double(), 0)[0].t().contiguous()
    _close(dw, ty @ tx.t().contiguous(), R.product_bound(ty, tx), ("dw", M, K, N))
    want, mags = dy.double().sum(0), dy.double().abs().sum(0)
    # 4 tokens, then 32 groups in four quarters, then the blocks of 128 in 32 chains: less than this many
    _close(db, want, (2 + 16 + 1 + M / 128 + 1) * R.F32 * mags + R.half_step(torch.bfloat16) * want.abs() * 1.001,
           ("db", M, K, N), many=False)
    again = S.fp8_backward(K, N, dev, x, dy)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


def test_backward_parts():
    """Each gradient alone is the bits of all three; x or qt may be absent
    where nothing reads them."""
    g = torch.Generator(device="cuda").manual_seed(2)
    M, K, N = 200, 272, 400
    x, dy = _bf16(g, M, K), _bf16(g, M, N)
    _, dev = _layer(g, K, N)
    full = S.fp8_backward(K, N, dev, x, dy)
    dx, a, b = S.fp8_backward(K, N, dev, None, dy, need=(True, False, False))
    assert torch.equal(dx, full[0]) and a is None and b is None
    bare = {"q": dev["q"], "s": dev["s"]}
    _, dw, db = S.fp8_backward(K, N, bare, x, dy, need=(False, True, True))
    assert torch.equal(dw, full[1]) and torch.equal(db, full[2])
    assert torch.equal(S.fp8_backward(K, N, bare, None, dy, need=(False, False, True))[2], full[2])


def test_gradients_against_differences():
    """On whole numbers every quantizer is exact and the loss sum(dy y) is
    bilinear, so central differences with whole steps are the gradients."""
    g = torch.Generator(device="cuda").manual_seed(11)
    M, K, N = 140, 144, 160
    x = torch.randint(-4, 5, (M, K), device="cuda", generator=g).to(torch.bfloat16)
    w = torch.randint(-4, 5, (N, K), device="cuda", generator=g).float()
    dy = torch.randint(-3, 4, (M, N), device="cuda", generator=g).to(torch.bfloat16)
    dev = S.fp8_pack(w)
    dx, dw, db = S.fp8_backward(K, N, dev, x, dy)

    def loss(xx, ww):   # |y| <= 144 * 16 + ... is rounded to bf16: use the exact float64 of the same product
        return (dy.double() * (xx.double() @ ww.double().t().contiguous())).sum()

    for i, j in [(0, 0), (139, 143), (64, 7), (3, 100)]:
        e = torch.zeros_like(x)
        e[i, j] = 1
        assert float((loss(x + e, w) - loss(x - e, w)) / 2) == pytest.approx(float(dx[i, j]), abs=0.5 * 2 ** -7 * abs(float(dx[i, j])))
    for i, j in [(0, 0), (159, 143), (64, 7), (3, 100)]:
        e = torch.zeros_like(w)
        e[i, j] = 1
        assert float((loss(x, w + e) - loss(x, w - e)) / 2) == pytest.approx(float(dw[i, j]), abs=0.5 * 2 ** -7 * abs(float(dw[i, j])))
    assert torch.equal(db, dy.float().sum(0).to(torch.bfloat16))
    assert torch.equal(dx, (dy.double() @ w.double()).to(torch.bfloat16))
    assert torch.equal(dw, (dy.double().t().contiguous() @ x.double()).to(torch.bfloat16))


def test_empty():
    g = torch.Generator(device="cuda").manual_seed(1)
    _, dev = _layer(g, 144, 48)
    x, dy = torch.empty(0, 144, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 48, dtype=torch.bfloat16, device="cuda")
    assert S.fp8_forward(144, 48, dev, x).shape == (0, 48)
    assert S.fp8_norm_forward(144, 48, dev, x).shape == (0, 48)
    for grads in (torch.bfloat16, torch.float32):
        dx, dw, db = S.fp8_backward(144, 48, dev, x, dy)
        assert dx.shape == (0, 144) and bool((dw == 0).all()) and bool((db == 0).all())


def test_training_step_stream_and_graph():
    """Norm, FP8 layer and their gradients as a step runs them: eagerly, on
    another stream, and captured and replayed with new inputs."""
    g = torch.Generator(device="cuda").manual_seed(9)
    M, K, N = 384, 272, 528
    w = torch.randn(N, K, device="cuda", generator=g) / K ** 0.5
    lin = S.Fp8Linear(w, torch.zeros(N, device="cuda"))
    x, dy = _bf16(g, M, K), _bf16(g, M, N)
    nw, nb = _bf16(g, 2, K, scale=0.2, outliers=False), _bf16(g, 2, K, outliers=False)

    def step(stream=None):
        lin.update(w, stream=stream)
        y, mean, rstd = lin.after_norm(x, nw, nb, one_plus=True, rows_per_group=192, stats=True, stream=stream)
        h, _, _ = S.layer_norm_forward(x, nw, nb, one_plus=True, rows_per_group=192, stream=stream)
        dh, dw, db = lin.backward(h, dy, stream=stream)
        return (y, dw, db) + S.layer_norm_backward(dh, x, mean, rstd, nw, one_plus=True, rows_per_group=192, stream=stream)

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        x.copy_(_bf16(g, M, K))
        w.mul_(1.25)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(kept, step())), k


def test_modulated_norm_between_the_w4a16_and_w4a4_layers():
    """The adaptive norm of a block: the W4A16 modulation layer's output split
    into shift and scale, the norm, and a W4A4 layer on its output."""
    import numpy as np
    from bit_svdquant_diffusion_amd import synth
    from oracle import svdq_oracle as O
    from tests import gpu_cases as C
    spec = synth.LayerSpec("norm_w4a4", 320, 512, 256, 16, "int4", 4)
    lay = synth.make_layer(spec)
    ref = O.pack(lay.w_lin, lay.bias, np.abs(lay.x).max(axis=0), spec.rank, "int4")
    layer = S.Layer(spec.K, spec.N, spec.rank, "int4")
    lin = S.SVDQLinear(layer, S.quantize_residual(layer, lay.w_lin, lay.bias, ref["mu"], O.bf16_to_bits(ref["l1"]),
                                                  O.bf16_to_bits(ref["l2"])))
    rng = np.random.default_rng(0)
    aw = (0.02 * rng.standard_normal((6 * spec.K, 128))).astype(np.float32)
    host, _, _ = S.awq_pack(aw, None, rng.standard_normal((8, 128)).astype(np.float32), alpha=0.5)
    cond = torch.from_numpy(rng.standard_normal((2, 128)).astype(np.float32)).cuda().to(torch.bfloat16)
    mod = S.awq_forward(128, 6 * spec.K, S.awq_to_device(host), cond)
    x = torch.from_numpy(lay.x_bits.view(np.int16)).cuda().view(torch.bfloat16)
    h, mean, rstd = S.layer_norm_forward(x, mod[:, spec.K:2 * spec.K], mod[:, :spec.K], one_plus=True, rows_per_group=160)
    want = R.layer_norm(x, mod[:, spec.K:2 * spec.K], mod[:, :spec.K], 1e-6, True, 160)[0]
    assert bool(((h.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all())
    y = lin(h)
    C.check_y(C.bf16_tensor_to_f32(y), O.forward(ref, h.float().cpu().numpy()), "norm then w4a4")


# few outputs over many channels (their runs are joined), the last run short,
# and persistent workgroups with several of the largest tiles
@pytest.mark.parametrize("M,K,N", [(17, 4112, 80), (33, 12288, 64), (64, 2064, 1040), (130, 8208, 272), (20, 65536, 16),
                                   (300, 1936, 144), (4090, 272, 4080), (8200, 144, 8208)])
def test_forward_runs_and_tiles(M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    x = _bf16(g, M, K)
    _, dev = _layer(g, K, N, transposed=False)
    need = S.fp8_workspace_bytes(K, N, M)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    y = S.fp8_forward(K, N, dev, x, workspace=ws[:need])
    assert bool((ws[need:] == 0xFF).all())
    a, w = R.q8(x.double())[0], _weight(dev, K, N)
    bias = dev["bias"].double()
    _close(y, a @ w.t().contiguous() + bias, R.product_bound(a, w, bias), (M, K, N))
    assert torch.equal(y, S.fp8_forward(K, N, dev, x))


@pytest.mark.parametrize("M,K,N", [(4112, 80, 48), (40, 48, 4112), (300, 4080, 4096)])
def test_backward_runs_and_tiles(M, K, N):
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    x, dy = _bf16(g, M, K), _bf16(g, M, N, scale=1e-3)
    _, dev = _layer(g, K, N)
    need = S.fp8_backward_workspace_bytes(K, N, M)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    dx, dw, _ = S.fp8_backward(K, N, dev, x, dy, workspace=ws[:need])
    assert bool((ws[need:] == 0xFF).all())
    w = _weight(dev, K, N)
    a = R.q8(dy.double())[0]
    _close(dx, a @ w, R.product_bound(a, w.t().contiguous()), ("dx", M, K, N))
    ty, tx = R.q8(dy.double(), 0)[0].t().contiguous(), R.q8(x.double(), 0)[0].t().contiguous()
    _close(dw, ty @ tx.t().contiguous(), R.product_bound(ty, tx), ("dw", M, K, N))


@pytest.mark.parametrize("M", [1, 2, 16])
def test_norm_forward_of_a_few_tokens_is_the_composition(M):
    g = torch.Generator(device="cuda").manual_seed(M)
    K, N = 528, 272
    x = _bf16(g, M, K)
    _, dev = _layer(g, K, N, transposed=False)
    w = torch.randn(K, device="cuda", generator=g).to(torch.bfloat16)
    h = S.layer_norm_forward(x, w)[0]
    assert torch.equal(S.fp8_norm_forward(K, N, dev, x, w), S.fp8_forward(K, N, dev, h))


def test_inline_limit():
    """Both sides of the size up to which one kernel quantizes its own tokens."""
    g = torch.Generator(device="cuda").manual_seed(3)
    N = 48
    for M, K in [(16, 3072), (16, 3088), (1, 49152), (1, 49168), (3, 16384), (3, 16400)]:
        x = _bf16(g, M, K)
        _, dev = _layer(g, K, N, transposed=False)
        assert (S.fp8_workspace_bytes(K, N, M) == 0) == (M * (-(-K // 128) * 128) <= 49152)
        y = S.fp8_forward(K, N, dev, x)
        a, w = R.q8(x.double())[0], _weight(dev, K, N)
        bias = dev["bias"].double()
        _close(y, a @ w.t().contiguous() + bias, R.product_bound(a, w, bias), (M, K, N))


def test_layer_refusals():
    g = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randn(64, 128, device="cuda", generator=g)
    lin = S.Fp8Linear(w)
    x = _bf16(g, 4, 128)
    for bad in (torch.randn(48, 128, device="cuda"), torch.randn(128, 64, device="cuda")):
        with pytest.raises(ValueError):
            lin.update(bad)
    with pytest.raises(ValueError):
        S.fp8_pack(w, torch.zeros(65, device="cuda"))
    ws = torch.empty(2, S.fp8_workspace_bytes(128, 64, 40), dtype=torch.uint8, device="cuda").t()
    with pytest.raises(ValueError):
        S.fp8_forward(128, 64, lin.dev, _bf16(g, 40, 128), workspace=ws)
    half = dict(lin.dev, bias=torch.zeros(64, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        S.fp8_forward(128, 64, half, x)
    for call in (lambda: lin(x.float()), lambda: lin(x[:, :112]), lambda: lin(x.t()), lambda: lin(x, y=x),
                 lambda: lin.backward(x, x), lambda: lin.after_norm(x, torch.ones(128, device="cuda").expand(2, 128))):
        with pytest.raises(ValueError):
            call()
    dy = _bf16(g, 4, 64)
    with pytest.raises(S.SvdqError):   # the input's gradient needs the transposed codes
        S.Fp8Linear(w, trainable=False).backward(x, dy)
    with pytest.raises(S.SvdqError):   # 16-byte alignment
        odd = _bf16(g, 5 * 128 + 1)[1:].view(5, 128)
        lin(odd)


def test_runs_in_graphs_and_on_two_streams():
    """Runs of channels (their tiles take tickets in the workspace): two graphs
    that share a workspace, replayed in turn with eager calls between, and two
    streams at once with workspaces of their own."""
    g = torch.Generator(device="cuda").manual_seed(6)
    M, K, N = 40, 8208, 272
    layers = [_layer(g, K, N, transposed=False)[1] for _ in range(2)]
    xs = [_bf16(g, M, K) for _ in range(2)]
    want = [S.fp8_forward(K, N, layers[i], xs[i]) for i in range(2)]
    ws = torch.empty(S.fp8_workspace_bytes(K, N, M), dtype=torch.uint8, device="cuda").fill_(0xFF)
    ys = [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            S.fp8_forward(K, N, layers[i], xs[i], y=ys[i], workspace=ws)
        graphs.append(graph)
    for k in range(4):
        for i in range(2):
            ys[i].zero_()
            graphs[i].replay()
            again = S.fp8_forward(K, N, layers[1 - i], xs[1 - i], workspace=ws)
            torch.cuda.synchronize()
            assert torch.equal(ys[i], want[i]) and torch.equal(again, want[1 - i]), (k, i)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(5):
        got = [S.fp8_forward(K, N, layers[i], xs[i], stream=streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k

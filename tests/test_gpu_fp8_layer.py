"""The FP8 layer as a program keeps it (MI355X only): its buffers over
updates, graphs and streams."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S

pytestmark = pytest.mark.gpu


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_bias_is_the_layers_own_buffer(dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(48, 64, device="cuda", generator=g)
    b = torch.randn(48, device="cuda", generator=g).to(dtype)
    dev = S.fp8_pack(w, b)
    want = b.to(torch.bfloat16).clone()
    assert dev["bias"].dtype == torch.bfloat16 and torch.equal(dev["bias"], want)
    b.fill_(9.0)   # the caller's, not the layer's
    assert torch.equal(dev["bias"], want)
    held = dict(dev)
    b2 = torch.randn(96, device="cuda", generator=g).to(dtype)[::2]   # strided
    S.fp8_pack(w * 2, b2, out=dev)
    assert all(dev[k] is held[k] for k in held) and torch.equal(dev["bias"], b2.to(torch.bfloat16))
    S.fp8_pack(w, out=dev)   # without a bias the layer keeps its own
    assert dev["bias"] is held["bias"] and torch.equal(dev["bias"], b2.to(torch.bfloat16))
    p = torch.nn.Parameter(b.float())
    S.fp8_pack(w, p, out=dev)   # a parameter's values, not its graph
    assert dev["bias"] is held["bias"] and not dev["bias"].requires_grad and bool((dev["bias"] == 9).all())
    lin = S.Fp8Linear(w)
    assert lin.dev["bias"] is None
    lin.update(w, p)
    assert torch.equal(lin.dev["bias"], held["bias"])


def test_a_refused_pack_changes_nothing():
    g = torch.Generator(device="cuda").manual_seed(2)
    w, b = torch.randn(48, 64, device="cuda", generator=g), torch.randn(48, device="cuda", generator=g)
    dev = S.fp8_pack(w, b)
    held, kept = dict(dev), {k: v.clone() for k, v in dev.items()}
    odd = torch.randn(48 * 64 + 1, device="cuda", generator=g)[1:].view(48, 64)   # not 16-byte aligned
    for call in (lambda: S.fp8_pack(w, b.cpu(), out=dev), lambda: S.fp8_pack(w, torch.zeros(47, device="cuda"), out=dev),
                 lambda: S.fp8_pack(torch.randn(48, 80, device="cuda"), b + 1, out=dev),
                 lambda: S.fp8_pack(w.double(), b + 1, out=dev), lambda: S.fp8_pack(odd, b + 1, out=dev)):
        with pytest.raises((ValueError, S.SvdqError)):
            call()
        torch.cuda.synchronize()
        assert all(dev[k] is held[k] and torch.equal(dev[k], kept[k]) for k in held)


@pytest.mark.parametrize("M", [3, 100])
def test_captured_forward_after_updates_of_weight_and_bias(M):
    """A graph of the layer reads what the last update wrote, on the current
    stream or another."""
    g = torch.Generator(device="cuda").manual_seed(3)
    K, N = 272, 144
    w, b = torch.randn(N, K, device="cuda", generator=g) / 16, torch.randn(N, device="cuda", generator=g)
    lin = S.Fp8Linear(w, b.to(torch.bfloat16))
    x = _bf16(g, M, K)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    lin(x, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin(x, y=y)
    side = torch.cuda.Stream()
    for k in range(4):
        w2, b2 = w * (k + 2), (b * (k + 2)).to(torch.bfloat16 if k % 2 else torch.float32)
        side.wait_stream(torch.cuda.current_stream())
        lin.update(w2, b2, stream=side if k >= 2 else None)
        torch.cuda.current_stream().wait_stream(side)
        filler = torch.full((1 << 12,), 77.0, dtype=torch.bfloat16, device="cuda")   # would take a released bias's place
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        fresh = S.Fp8Linear(w2, b2)
        assert torch.equal(y, fresh(x)) and torch.equal(y, lin(x)), k
        assert bool((filler == 77).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_captured_update_of_weight_and_bias(dtype):
    g = torch.Generator(device="cuda").manual_seed(4)
    M, K, N = 40, 144, 272
    w, b = torch.randn(N, K, device="cuda", generator=g), torch.randn(N, device="cuda", generator=g).to(dtype)
    lin, x = S.Fp8Linear(w, b), _bf16(g, M, K)
    lin(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.update(w, b)
        y = lin(x)
    for k in range(3):
        w.mul_(1.5)
        b.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        kept = y.clone()
        assert torch.equal(kept, S.Fp8Linear(w, b)(x)) and torch.equal(kept, lin(x)), k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_infinities_and_nan_of_a_weight_stay_in_their_channel(dtype):
    """A weight that is not finite becomes the NaN code; the other values of
    its 128 x 128 block keep the codes of a block without it (they would all
    be zeros under a scale for infinity), so other channels keep their outputs."""
    g = torch.Generator(device="cuda").manual_seed(5)
    K, N = 272, 400
    w = (torch.randn(N, K, device="cuda", generator=g) / 16).to(dtype)
    bad = [(3, 5, float("inf")), (140, 130, float("nan")), (399, 271, float("-inf"))]
    clean = w.clone()
    for n, k, v in bad:
        w[n, k], clean[n, k] = v, 0
    a, b = S.fp8_pack(w), S.fp8_pack(clean)
    assert torch.equal(a["s"], b["s"]) and torch.equal(a["st"], b["st"])
    for n, k, _ in bad:
        assert int(a["q"][n, k]) & 0x7F == 0x7F and int(a["qt"][k, n]) & 0x7F == 0x7F
        a["q"][n, k] = a["qt"][k, n] = 0
    assert torch.equal(a["q"], b["q"]) and torch.equal(a["qt"], b["qt"])
    for M in (3, 70):
        x = _bf16(g, M, K)
        y, want = S.Fp8Linear(w)(x), S.Fp8Linear(clean)(x)
        rows = torch.zeros(N, dtype=torch.bool, device="cuda")
        rows[[n for n, _, _ in bad]] = True
        assert bool(y[:, rows].isnan().all()) and torch.equal(y[:, ~rows], want[:, ~rows]), M


def test_a_weight_block_without_a_finite_value():
    w = torch.full((128, 256), float("nan"), device="cuda")
    w[:, 128:] = 1
    dev = S.fp8_pack(w)
    assert bool((dev["q"][:, :128] & 0x7F == 0x7F).all()) and dev["s"][0, :2].tolist() == [1, 127 - 8]
    assert bool((dev["q"][:, 128:].view(torch.float8_e4m3fn).float() == 256).all())

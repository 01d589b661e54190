"""A transformer block run and trained with the library's calls (MI355X only):
modulated layer norm, FP8 projections, rotary positions, attention over text
and image tokens, gated residual with the next norm, MLP. Every call of the run
is held to the float64 form of what it computes, on the inputs that it had in
the run; and a torch.autograd.Function made of the calls has their gradients."""
import pytest

torch = pytest.importorskip("torch")

import bit_svdquant_diffusion_amd as S
from tests import block_reference as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
B, L, TEXT, C, H, HK, D = 2, 333, 60, 512, 8, 4, 64
PAIRS = [4, 14, 14]


class Block:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)   # noqa: E731
        lin = lambda n, k: S.Fp8Linear(rnd(n, k) / k ** 0.5, 0.1 * rnd(n))   # noqa: E731
        self.qkv, self.out, self.up, self.down = lin((H + 2 * HK) * D, C), lin(C, H * D), lin(4 * C, C), lin(C, 4 * C)
        self.mod = (0.3 * rnd(B, 7 * C)).to(BF)   # shifts, scales and gates side by side, as a modulation layer leaves them
        self.post = rnd(C).mul_(0.1).to(BF).expand(B, C).contiguous()
        self.freqs = S.rope_frequencies(PAIRS)
        at = torch.arange(L, device="cuda") - TEXT
        self.pos = torch.stack([torch.zeros_like(at), at // 17, at % 17], 1).clamp(min=0).to(torch.int32)
        length = torch.tensor([[20], [TEXT]], device="cuda")
        self.mask = (torch.arange(L, device="cuda")[None] < length) | (torch.arange(L, device="cuda")[None] >= TEXT)
        self.x = rnd(B * L, C).to(BF)
        self.dy, self.ds = rnd(B * L, C).to(BF), rnd(B * L, C).to(BF)

    def part(self, i):
        return self.mod[:, i * C:(i + 1) * C]

    def forward(self, x, mod=None):
        t = {"x": x}
        p = self.part if mod is None else lambda i: mod[:, i * C:(i + 1) * C]
        t["n"], t["mean"], t["rstd"] = S.layer_norm_forward(x, p(1), p(0), one_plus=True, rows_per_group=L)
        t["qkv"] = self.qkv(t["n"]).view(B, L, H + 2 * HK, D)
        q, k, t["v"] = t["qkv"].split([H, HK, HK], 2)
        t["q"], t["k"] = S.rope(q, k, self.pos, self.freqs, PAIRS)
        t["o"], t["lse"] = S.attention_forward(t["q"], t["k"], t["v"], key_mask=self.mask)
        t["h"] = self.out(t["o"].view(B * L, H * D))
        t["s"], t["y"], t["stats"] = S.residual_norm_forward(x, t["h"], p(2), p(4), p(3), one_plus=True, rows_per_group=L)
        t["u"] = self.up(t["y"])
        t["a"] = torch.nn.functional.gelu(t["u"].float()).to(BF)
        t["h2"] = self.down(t["a"])
        t["s2"], t["y2"], t["stats2"] = S.residual_norm_forward(t["s"], t["h2"], p(5), p(6), None, post_weight=self.post, kind="rms",
                                                                one_plus=True, rows_per_group=L)
        return t

    def backward(self, t, dy, ds, mod=None):
        p = self.part if mod is None else lambda i: mod[:, i * C:(i + 1) * C]
        d = {}
        d["s"], d["h2"], g5, g6, _, d["post"] = S.residual_norm_backward(
            dy, t["s2"], t["h2"], t["stats2"], p(5), p(6), post_weight=self.post, ds=ds, kind="rms", one_plus=True, rows_per_group=L)
        d["a"], _, _ = self.down.backward(t["a"], d["h2"])
        u = t["u"].float().requires_grad_()
        with torch.enable_grad():
            d["u"] = torch.autograd.grad(torch.nn.functional.gelu(u), u, d["a"].float())[0].to(BF)
        d["y"], _, _ = self.up.backward(t["y"], d["u"])
        d["x1"], d["h"], g2, g4, g3, _ = S.residual_norm_backward(d["y"], t["s"], t["h"], t["stats"], p(2), p(4), ds=d["s"],
                                                                  one_plus=True, rows_per_group=L)
        d["o"], _, _ = self.out.backward(t["o"].view(B * L, H * D), d["h"])
        d["qkv"] = torch.empty_like(t["qkv"])
        dq, dk, dv = d["qkv"].split([H, HK, HK], 2)
        d["q"], d["k"], d["v"] = S.attention_backward(d["o"].view(B, L, H, D), t["q"], t["k"], t["v"], t["o"], t["lse"],
                                                      key_mask=self.mask, dv=dv)
        S.rope(d["q"], d["k"], self.pos, self.freqs, PAIRS, inverse=True, q_out=dq, k_out=dk)
        d["n"], _, _ = self.qkv.backward(t["n"], d["qkv"].view(B * L, -1))
        d["x0"], g1, g0 = S.layer_norm_backward(d["n"], t["x"], t["mean"], t["rstd"], p(1), one_plus=True, rows_per_group=L)
        d["x"] = d["x0"] + d["x1"]
        d["mod"] = torch.cat([g0, g1, g2, g3, g4, g5, g6], 1)
        return d


def test_every_call_of_the_run():
    m = Block()
    t = m.forward(m.x)
    q, k, _ = t["qkv"].split([H, HK, HK], 2)
    R.check(t["q"], R.rope(q, m.pos, m.freqs, PAIRS, True, False), "q")
    R.check(t["k"], R.rope(k, m.pos, m.freqs, PAIRS, True, False), "k")
    ref = R.attention(t["q"], t["k"], t["v"], m.mask, False, D ** -0.5)
    R.check(t["o"], ref["o"], "o")
    R.check(t["lse"], ref["lse"], "lse")
    ref = R.residual_norm(t["x"], t["h"], m.part(2), m.part(4), m.part(3), None, 1.0, 1e-6, "layer", False, True, L, s=t["s"])
    R.check(t["s"], ref["s"], "s")
    R.check(t["y"], ref["y"], "y")
    ref = R.residual_norm(t["s"], t["h2"], m.part(5), m.part(6), None, m.post, 1.0, 1e-6, "rms", True, True, L, s=t["s2"])
    R.check(t["s2"], ref["s"], "s2")
    R.check(t["y2"], ref["y"], "y2")
    d = m.backward(t, m.dy, m.ds)
    ref = R.residual_norm_grad(m.dy, m.ds, t["s2"], t["h2"], list(t["stats2"]), m.part(5), m.part(6), m.post, 1.0, "rms", True, True,
                               L, B, BF)
    for got, name in ((d["s"], "dx"), (d["h2"], "dh"), (d["post"], "dpost"), (d["mod"][:, 5 * C:6 * C], "dgate"),
                      (d["mod"][:, 6 * C:], "dweight")):
        R.check(got, ref[name], name + " after the MLP")
    ref = R.residual_norm_grad(d["y"], d["s"], t["s"], t["h"], list(t["stats"]), m.part(2), m.part(4), None, 1.0, "layer", False, True,
                               L, B, BF)
    for got, name in ((d["x1"], "dx"), (d["h"], "dh"), (d["mod"][:, 2 * C:3 * C], "dgate"), (d["mod"][:, 3 * C:4 * C], "dbias"),
                      (d["mod"][:, 4 * C:5 * C], "dweight")):
        R.check(got, ref[name], name + " after the attention")
    ref = R.attention(t["q"], t["k"], t["v"], m.mask, False, D ** -0.5, (d["o"].view(B, L, H, D), t["o"], t["lse"]))
    for name in "qkv":
        R.check(d[name], ref["d" + name], "d" + name)
    dq, dk, _ = d["qkv"].split([H, HK, HK], 2)
    R.check(dq, R.rope(d["q"], m.pos, m.freqs, PAIRS, True, True), "dq turned back")
    R.check(dk, R.rope(d["k"], m.pos, m.freqs, PAIRS, True, True), "dk turned back")
    # padded text keys take no part
    assert not bool(d["k"][0, 20:TEXT].any()) and not bool(d["v"][0, 20:TEXT].any())


class _Step(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, mod, m):
        t = m.forward(x, mod)
        ctx.t, ctx.m, ctx.mod = t, m, mod
        return t["y2"], t["s2"]

    @staticmethod
    def backward(ctx, dy, ds):
        d = ctx.m.backward(ctx.t, dy.contiguous(), ds.contiguous(), ctx.mod)
        return d["x"], d["mod"], None


def test_in_an_autograd_function():
    m = Block(1)
    x, mod = m.x.clone().requires_grad_(), m.mod.clone().requires_grad_()
    y, s = _Step.apply(x, mod, m)
    torch.autograd.backward([y, s], [m.dy, m.ds])
    want = m.backward(m.forward(m.x), m.dy, m.ds)
    assert torch.equal(x.grad, want["x"]) and torch.equal(mod.grad, want["mod"])


def test_captured_and_replayed():
    m = Block(2)
    keys = ("y2", "s2", "lse")
    want_t = m.forward(m.x)
    want_d = m.backward(want_t, m.dy, m.ds)
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.forward(m.x)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        t = m.forward(m.x)
    for _ in range(3):
        for k in keys:
            t[k].zero_()
        eager = m.backward(want_t, m.dy, m.ds)   # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t[k], want_t[k]) for k in keys)
        assert torch.equal(eager["x"], want_d["x"]) and torch.equal(eager["mod"], want_d["mod"])

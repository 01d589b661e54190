"""Plain float64 forms of the operators between a block's linears (gated
residual with its norms, rotary positions, attention) and their gradients,
with a bound for what a computation in 32 bits may be off by. A `Bound` value
is a pair (value, error) of float64 tensors.

Tolerances. u = 2^-24 is half a step of an fp32 operation, eps(t) half a step of
the type t. A sum over a row of a norm takes at most CHAIN additions one after
the other; sums over rows or keys are bounded by their length. Each operation
adds its half step to first order, the last rounding eps(type)."""
import math

import torch

U = 2.0 ** -24
CHAIN = 48   # 8 elements in a lane, 6 steps over the wave, 16 waves, the rest in reserve


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(value, error, dtype):
    """The bound after the rounding to the type (fp16: its subnormals' step)."""
    return error * (1 + half_step(dtype)) + half_step(dtype) * value.abs() + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -140)


def norm(v, kind, eps):
    """(norm(v), its error, mean, its error, rstd, its relative error) of float64 rows."""
    n = v.shape[1]
    mean = v.mean(1) if kind == "layer" else torch.zeros(v.shape[0], dtype=v.dtype, device=v.device)
    e_mean = (CHAIN + 2) * U * v.abs().mean(1) if kind == "layer" else torch.zeros_like(mean)
    off = v - mean[:, None]
    rstd = ((off * off).sum(1) / n + eps).rsqrt()
    e_rstd = (CHAIN / 2 + 6) * U + rstd.square() * e_mean.square()
    hat = off * rstd[:, None]
    return hat, rstd[:, None] * e_mean[:, None] + hat.abs() * (e_rstd[:, None] + 3 * U), mean, e_mean, rstd, e_rstd


def of_rows(p, rows, rows_per_group, add=0.0, fill=1.0):
    """A parameter's value for each row ([C] or [groups][C], or None)."""
    if p is None:
        return torch.full((rows, 1), fill, dtype=torch.float64)
    p = p.double() if p.dim() == 2 else p.double()[None]
    return p[torch.arange(rows, device=p.device) // rows_per_group] + add


def residual_norm(x, h, gate, weight, bias, post, alpha, eps, kind, post_norm, one_plus, rpg, s=None):
    """{name: (value, error)} of s, y and the statistics. y is the norm of the
    given s (what the device wrote), or of the rounded reference."""
    rows, one = x.shape[0], 1.0 if one_plus else 0.0
    dev = x.device
    g = of_rows(gate, rows, rpg).to(dev)
    hn, e_hn = h.double(), torch.zeros_like(h, dtype=torch.float64)
    out = {}
    if post_norm:
        hat, e_hat, pm, epm, pr, epr = norm(hn, kind, eps)
        gp = of_rows(post, rows, rpg, one).to(dev)
        hn, e_hn = hat * gp, e_hat * gp.abs() + 3 * U * (hat * gp).abs()
        out["post"] = (pm, epm, pr, epr)
    ref = alpha * x.double() + g * hn
    err = g.abs() * e_hn + 3 * U * ((alpha * x.double()).abs() + (g * hn).abs())
    out["s"] = (ref, rounded(ref, err, x.dtype))
    s = ref.to(x.dtype) if s is None else s
    hat, e_hat, m, em, r, er = norm(s.double(), kind, eps)
    gain, shift = of_rows(weight, rows, rpg, one).to(dev), of_rows(bias, rows, rpg, 0.0, 0.0).to(dev)
    y = hat * gain + shift
    out["y"] = (y, rounded(y, gain.abs() * e_hat + 3 * U * (hat * gain).abs() + U * shift.abs(), x.dtype))
    out["norm"] = (m, em, r, er)
    return out


def _through(d, e_d, hat, rstd, kind):
    """A norm's gradient for d (with error e_d), and its error."""
    c1 = d.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(d[:, :1])
    c2 = (d * hat).mean(1, keepdim=True)
    value = rstd * (d - c1 - hat * c2)
    err = e_d + (e_d.mean(1, keepdim=True) if kind == "layer" else 0.0) + hat.abs() * (e_d * hat.abs()).mean(1, keepdim=True)
    err = err + (CHAIN + 6) * U * d.abs().mean(1, keepdim=True) + hat.abs() * (CHAIN + 12) * U * (d * hat).abs().mean(1, keepdim=True)
    return value, rstd * (err + 6 * U * (d.abs() + c1.abs() + (hat * c2).abs()))


def residual_norm_grad(dy, ds, s, h, stats, gate, weight, post, alpha, kind, post_norm, one_plus, rpg, groups, gdtype):
    """{name: (value, error)} of dx, dh and the parameters' gradients
    [groups][C], from the statistics that the forward left."""
    rows, one, dev = s.shape[0], 1.0 if one_plus else 0.0, s.device
    st = [v.double()[:, None] for v in stats]
    zero = torch.zeros(rows, 1, dtype=torch.float64, device=dev)
    n = 2 if kind == "layer" else 1
    mean, rstd = (st[0], st[1]) if kind == "layer" else (zero, st[0])
    shat = (s.double() - mean) * rstd
    g, gain = of_rows(gate, rows, rpg).to(dev), of_rows(weight, rows, rpg, one).to(dev)
    dyd = dy.double()
    d = dyd * gain
    t, e_t = _through(d, 2 * U * d.abs(), shat, rstd, kind)
    along = ds.double() if ds is not None else torch.zeros_like(t)
    t = t + along
    e_t = e_t + 2 * U * (t.abs() + along.abs())
    out = {"dx": (alpha * t, rounded(alpha * t, abs(alpha) * e_t + 2 * U * (alpha * t).abs(), s.dtype))}
    e, e_e = t * g, e_t * g.abs() + 2 * U * (t * g).abs()
    hn, e_hn = h.double(), torch.zeros_like(t)
    dh, e_dh = e, e_e
    sums = {}
    if post_norm:
        hmean, hrstd = (st[n], st[n + 1]) if kind == "layer" else (zero, st[n])
        hhat = (hn - hmean) * hrstd
        gp = of_rows(post, rows, rpg, one).to(dev)
        hn, e_hn = hhat * gp, 4 * U * (hhat * gp).abs()
        sums["dpost"] = (e * hhat, e_e * hhat.abs() + 3 * U * (e * hhat).abs())
        f, e_f = e * gp, e_e * gp.abs() + 2 * U * (e * gp).abs()
        dh, e_dh = _through(f, e_f, hhat, hrstd, kind)
    out["dh"] = (dh, rounded(dh, e_dh, s.dtype))
    sums["dgate"] = (t * hn, e_t * hn.abs() + t.abs() * e_hn + 3 * U * (t * hn).abs())
    sums["dweight"] = (dyd * shat, 4 * U * (dyd * shat).abs())
    sums["dbias"] = (dyd, torch.zeros_like(dyd))
    for name, (v, err) in sums.items():
        c = v.shape[1]
        val, bound = (torch.zeros(groups, c, dtype=torch.float64, device=dev) for _ in range(2))
        for i in range(groups):
            part = slice(i * rpg, min((i + 1) * rpg, rows))
            val[i] = v[part].sum(0)
            bound[i] = err[part].sum(0) + (v[part].shape[0] + 8) * U * v[part].abs().sum(0)
        out[name] = (val, rounded(val, bound, gdtype))
    return out


def rope(x, positions, freqs, pairs, interleaved, inverse):
    """(value, error) of x [B][L][H][D] turned."""
    axis = torch.repeat_interleave(torch.arange(len(pairs)), torch.tensor(pairs)).to(x.device)
    p = positions.double() if positions.dim() == 3 else positions.double()[None]
    angle = p[..., axis] * freqs * (-1.0 if inverse else 1.0)
    c, s = angle.cos()[:, :, None], angle.sin()[:, :, None]
    n, y = sum(pairs), x.double().clone()
    e = torch.zeros_like(y)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    u, v = x.double()[..., a], x.double()[..., b]
    y[..., a], y[..., b] = u * c - v * s, u * s + v * c
    # the turns' fraction is rounded once (2 pi 2^-26 < 1.6 U), cosine and sine
    # to 2 U, two products and a sum; the angle itself to a few steps of 64 bits
    off = (u.abs() + v.abs()) * (6 * U + 4 * 2.0 ** -53 * angle.abs()[:, :, None])
    e[..., a], e[..., b] = off, off
    err = torch.where(e > 0, rounded(y, e, x.dtype), torch.zeros_like(e))   # what passes through keeps its bits
    return y, err


def visible(Lq, Lk, causal, mask, device):
    see = torch.ones(Lq, Lk, dtype=torch.bool, device=device)
    if causal:
        see = torch.arange(Lk, device=device)[None] <= torch.arange(Lq, device=device)[:, None] + Lk - Lq
    return see if mask is None else see & mask.bool()[None]


def _scores(q, k, see, scale):
    """(scores, their error) of a head: a sum of D products in fp32, the scale
    and the difference from the maximum (or lse) in base 2."""
    s = torch.where(see, torch.mm(q, k.t().contiguous()) * scale, -math.inf)
    mag = torch.mm(q.abs(), k.abs().t().contiguous()) * abs(scale)
    return s, (q.shape[1] + 4) * U * mag


def attention(q, k, v, mask, causal, scale, grad=None, fine=False):
    """{name: (value, error)}: o and lse; with grad = (dout, o, lse) dq, dk and dv."""
    B, Lq, H, D = q.shape
    Lk, Hk, dt = k.shape[1], k.shape[2], q.dtype
    half, tiny = half_step(dt), dt == torch.float16
    if fine or D <= 32 or Lq * (H // Hk) <= 64 or Lk <= 64:   # probabilities and ds enter their products as two values, the second what the first's rounding left
        half = 1.01 * half * half
    dev = q.device

    def zeros(*shape):
        return [torch.zeros(*shape, dtype=torch.float64, device=dev) for _ in range(2)]
    o, lse, dq, dk, dv = zeros(B, Lq, H, D), zeros(B, H, Lq), zeros(B, Lq, H, D), zeros(B, Lk, Hk, D), zeros(B, Lk, Hk, D)
    mm = lambda a, b: torch.mm(a, b.contiguous())   # noqa: E731
    for b in range(B):
        see = visible(Lq, Lk, causal, None if mask is None else mask[b], dev)
        keep, live = see.any(0), see.any(1)   # what nothing sees, or sees nothing, does not count whatever it holds
        if grad is not None:
            top_v = v[b].double()[keep].abs().max().item() if bool(keep.any()) else 0.0
            top_do = grad[0][b].double()[live].abs().max().item() if bool(live.any()) else 0.0
        for h in range(H):
            kv = h * Hk // H
            q1 = torch.where(live[:, None], q[b, :, h].double(), 0.0)
            k1 = torch.where(keep[:, None], k[b, :, kv].double(), 0.0)
            v1 = torch.where(keep[:, None], v[b, :, kv].double(), 0.0)
            s, e_s = _scores(q1, k1, see, scale)
            if grad is None:
                m = s.amax(1, keepdim=True) if Lk else torch.full((Lq, 1), -math.inf, dtype=torch.float64, device=dev)
                p = torch.where(see, torch.exp(s - m.clamp(min=-1e300)), 0.0)
                l = p.sum(1, keepdim=True)
                lse[0][b, h] = (m + torch.log(l))[:, 0]
                p = p / l.clamp(min=1e-300)
                # a score's distance to the maximum costs its own rounding
                dist = torch.where(see, (s - m).abs() + 16, 0.0) * 2 * U
                e_p = p * (e_s + dist + 4 * U)
                e_l = e_p.sum(1, keepdim=True) + (Lk + 4) * U * live[:, None]
                lse[1][b, h] = e_l[:, 0] + 4 * U * lse[0][b, h].abs().clamp(max=1e30)
                o[0][b, :, h] = mm(p, v1)
                spread = mm(p * (half + (Lk + 8) * U) + e_p, v1.abs()) + e_l * mm(p, v1.abs())
                if tiny:
                    spread = spread + 2.0 ** -25 * (see.double() @ v1.abs()) * 1.0
                o[1][b, :, h] = rounded(o[0][b, :, h], spread, dt)
                continue
            dout, o1, l1 = grad
            do = torch.where(live[:, None], dout[b, :, h].double(), 0.0)
            p = torch.where(see, torch.exp(s - torch.where(live, l1[b, h].double(), 0.0)[:, None]), 0.0)
            # lse enters as the value that the product's accumulator starts with
            # (D / 16 further roundings of a sum that holds it)
            e_p = p * (half + e_s + torch.where(see, (s.abs() + l1[b, h].double().abs().clamp(max=1e30)[:, None]) * (4 + D / 16) * U, 0.0) + 4 * U)
            # A probability below 2^-126 is zero in fp32 (the exponential has no
            # subnormal results), and so is a ds: p is off by 2^-126 at most
            # beside its relative error, ds by that much of dp - delta and
            # 2^-126 of its own.
            e_p = e_p + see * 2.0 ** -126
            low = 2.0 ** -35 if tiny else 0.0
            dv[0][b, :, kv] += mm(p.t(), do)
            dv[1][b, :, kv] += mm(e_p.t() + low * see.t() + (Lq * H + 8) * U * p.t(), do.abs())
            delta = torch.where(live, (do * o1[b, :, h].double()).sum(1), 0.0)[:, None]
            dp = mm(do, v1.t())
            ds = p * (dp - delta)
            e_d = (D + 4) * U * (mm(do.abs(), v1.abs().t()) + (do * torch.where(live[:, None], o1[b, :, h].double(), 0.0)).abs().sum(1, keepdim=True))
            e_ds = p * e_d + e_p * (dp - delta).abs() + 4 * U * ds.abs() + see * 2.0 ** -126
            if tiny:   # the scaled ds: 2^-25 where the largest possible one is 2^14 at least
                e_ds = e_ds + see * 2.0 ** -39 * 2 * D * top_v * top_do
            dq[0][b, :, h] = mm(ds, k1) * scale
            dq[1][b, :, h] = rounded(dq[0][b, :, h], mm(e_ds + (Lk + 8) * U * ds.abs(), k1.abs()) * scale, dt)
            dk[0][b, :, kv] += mm(ds.t(), q1) * scale
            dk[1][b, :, kv] += mm(e_ds.t() + (Lq * H + 8) * U * ds.abs().t(), q1.abs()) * scale
    if grad is None:
        return {"o": o, "lse": lse}
    return {"dq": dq, "dk": (dk[0], rounded(dk[0], dk[1], dt)), "dv": (dv[0], rounded(dv[0], dv[1], dt))}


def check(got, want, what):
    """Every element within its bound; NaN and infinities in the same places."""
    value, error = want
    got = got.double()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    fine = torch.isfinite(value)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: not finite where the value is, or the other way round"
    assert torch.equal(got[~fine & ~value.isnan()], value[~fine & ~value.isnan()]), what
    off = (got - value).abs()[fine]
    bad = off > error[fine]
    if bool(bad.any()):
        worst = float((off / error[fine].clamp(min=1e-300)).max())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, up to {worst:.3g} times the bound")

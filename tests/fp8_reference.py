"""Layer norm and the FP8 linear in float64, written from their definitions:
no code of the library is used."""
import torch

# fp32 sums on the vector ALU: half a step per addition
F32 = 2.0 ** -24


def half_step(dtype):
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def round_e4m3(v):
    """Nearest E4M3 value (ties to even) of float64 values with |v| <= 448."""
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(exponent - 3)
    return torch.round(v / step) * step


def block_exponent(top):
    """The least e >= -126 with top 2^-e <= 448, by search from the estimate."""
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448)) + 2
    for _ in range(3):
        e = torch.where(top * torch.exp2(-(e - 1)) <= 448, e - 1, e)
    e = torch.where(top > 0, e, torch.full_like(e, -126.0))
    return e.clamp(min=-126.0)


def q8(v, axis=1):
    """(values, exponents) of float64 v quantized in blocks of 128 along axis."""
    if axis == 0:
        q, e = q8(v.t(), 1)
        return q.t(), e.t()
    out = torch.empty_like(v)
    es = []
    for at in range(0, v.shape[1], 128):
        b = v[:, at:at + 128]
        e = block_exponent(b.abs().amax(1, keepdim=True))
        out[:, at:at + 128] = round_e4m3(b * torch.exp2(-e)) * torch.exp2(e)
        es.append(e)
    return out, torch.cat(es, 1)


def q8_blocks(w):
    """(values, exponents) of a weight in 128 x 128 blocks."""
    out = torch.empty_like(w)
    n, k = -(-w.shape[0] // 128), -(-w.shape[1] // 128)
    es = torch.empty(n, k, dtype=torch.float64, device=w.device)
    for i in range(n):
        for j in range(k):
            b = w[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            e = block_exponent(b.abs().max())
            out[128 * i:128 * i + 128, 128 * j:128 * j + 128] = round_e4m3(b * torch.exp2(-e)) * torch.exp2(e)
            es[i, j] = e
    return out, es


def _eights(v):
    """The largest magnitude of each eight consecutive channels."""
    short = -v.shape[1] % 8
    if short:
        v = torch.cat([v, v.new_zeros(v.shape[0], short)], 1)
    return v.abs().view(v.shape[0], -1, 8).amax(2)


def product_bound(a, b, extra=0.0):
    """How far a bf16 output of a b^T (+ extra) may be off, per output. The
    matrix unit aligns the products of eight consecutive channels to the
    largest one's exponent and cuts each below 2^-13 of it (seen with pairs
    and fives of powers of two: 2^16 + 2^3 is exact, 2^16 + n 2^2 loses the
    2^2s), so an eight loses at most 7 2^-13 times its largest product, which
    is at most the product of the largest factors. Then fp32 additions: at
    most one per eight, each a step (2^-23) of at most the sum of magnitudes;
    the addition of extra; one rounding to bf16."""
    cut = 7 * 2.0 ** -13 * (_eights(a) @ _eights(b).t().contiguous())
    sums = (a.shape[1] / 8 + 2) * 2.0 ** -23 * (a.abs() @ b.abs().t().contiguous())
    exact = (a @ b.t().contiguous() + extra).abs()
    return (cut + sums + F32 * exact) * (1 + half_step(torch.bfloat16)) + half_step(torch.bfloat16) * exact


def layer_norm(x, weight, bias, eps, one_plus, rows_per_group):
    x = x.double()
    mean = x.mean(1)
    off = x - mean[:, None]
    rstd = 1 / torch.sqrt(off.square().mean(1) + eps)
    xhat = off * rstd[:, None]
    g = torch.arange(x.shape[0], device=x.device) // rows_per_group
    gain = torch.ones_like(x) if weight is None else weight.double()[g] + (1.0 if one_plus else 0.0)
    shift = torch.zeros_like(x) if bias is None else bias.double()[g]
    return xhat * gain + shift, mean, rstd, xhat, gain


def layer_norm_grad(dy, x, weight, eps, one_plus, rows_per_group, groups):
    dy = dy.double()
    _, mean, rstd, xhat, gain = layer_norm(x, weight, None, eps, one_plus, rows_per_group)
    d = dy * gain
    dx = rstd[:, None] * (d - d.mean(1, keepdim=True) - xhat * (d * xhat).mean(1, keepdim=True))
    g = torch.arange(x.shape[0], device=x.device) // rows_per_group
    dw = torch.zeros(groups, x.shape[1], dtype=torch.float64, device=x.device)
    db = torch.zeros_like(dw)
    for i in range(groups):
        dw[i] = (dy * xhat)[g == i].sum(0)
        db[i] = dy[g == i].sum(0)
    return dx, dw, db

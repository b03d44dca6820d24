"""fp64 CPU oracle of the row calls: norms of rows with their gradients, and
8-bit activation checkpoints. Plain torch in float64, from the definitions;
shares no code with the CUDA path."""
import torch

F64 = torch.float64


def norm_fwd(x, weight, bias, eps, center, base):
    """(y, mean, rstd) of rows x[..., D]; weight and bias broadcast against x."""
    x = x.to(F64)
    mean = x.mean(-1) if center else torch.zeros(x.shape[:-1], dtype=F64)
    dev = x - mean[..., None]
    rstd = (dev.square().mean(-1) + eps) ** -0.5
    y = dev * rstd[..., None]
    if weight is not None:
        y = y * (weight.to(F64) + base)
    if bias is not None:
        y = y + bias.to(F64)
    return y, mean, rstd


def norm_bwd(dy, x, mean, rstd, weight, bias, base):
    """(dx, dweight, dbias) at the statistics given; mean None: not centred."""
    dy, x, rstd = dy.to(F64), x.to(F64), rstd.to(F64)[..., None]
    xhat = (x - mean.to(F64)[..., None] if mean is not None else x) * rstd
    g = dy * (weight.to(F64) + base) if weight is not None else dy
    dx = g - xhat * (g * xhat).mean(-1, keepdim=True)
    if mean is not None:
        dx = dx - g.mean(-1, keepdim=True)

    def over_rows(t, p):
        if p is None:
            return None
        shape = (1,) * (t.dim() - p.dim()) + tuple(p.shape)
        return t.sum([i for i, n in enumerate(shape) if n == 1 and i < t.dim() - 1], keepdim=True).reshape(p.shape)

    return rstd * dx, over_rows(dy * xhat, weight), over_rows(dy, bias)


def pack(x):
    """(q int64 [..., D], e int64 [..., ceil(D/32)]) of finite or non-finite x."""
    x = x.to(F64)
    D = x.shape[-1]
    q = torch.zeros(x.shape, dtype=torch.int64)
    e = torch.zeros(tuple(x.shape[:-1]) + ((D + 31) // 32,), dtype=torch.int64)
    for b in range(e.shape[-1]):
        part = x[..., 32 * b:32 * b + 32]
        top = part.abs().amax(-1)                           # NaN where the block holds one
        fine = torch.isfinite(top)
        _, power = torch.frexp(torch.where(fine, top, torch.ones_like(top)))
        # top in [2^(power-1), 2^power): the exponent field of fp32 is power - 1 + 127
        eb = torch.where(fine & (top > 0), power.to(torch.int64) + 126, torch.full_like(power, 7).to(torch.int64))
        eb = torch.where(fine, eb.clamp(min=7), torch.full_like(eb, 255))
        e[..., b] = eb
        part = torch.where(fine[..., None], part, torch.zeros_like(part))
        q[..., 32 * b:32 * b + 32] = torch.round(part / torch.exp2(eb[..., None].to(F64) - 133)).clamp(-127, 127)
    return q, e


def unpack(q, e):
    step = torch.exp2(e.to(F64) - 133)
    step = torch.where(e == 255, torch.full_like(step, float("nan")), step)
    return q.to(F64) * step.repeat_interleave(32, -1)[..., :q.shape[-1]]

"""The row calls on the GPU against the fp64 oracle: norms forward and backward,
8-bit checkpoints, and both as a layer's training step uses them.

Tolerances. Every sum runs in fp32 over at most 16 channels a thread and 10
shuffle levels, so a row's sum is off by at most 26 roundings of 2^-24 of the
sum of magnitudes; with the scaling and the subtractions C = 64 roundings
cover each term. An output is rounded once more, by half a step of its type."""
import pytest
import torch

import dynamic_sparse_attention_dsv_gb300 as dsv
from oracle import rows_oracle as ora

from .rows_cases import (BF16, FP16, FP32, LAYOUTS, PARAMS, SHAPES, TYPES, guarded, half_step, inputs, lay,
                         outside_kept, params)

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
C = 64
EPS = 1e-6

#: every shape with every type pair; layout, parameters and centring vary along
CASES = [(shape, xt, yt, LAYOUTS[(i + 3 * j) % 4], PARAMS[(i + j) % 6], (i + j) % 3 != 0, float((i // 2 + j) % 2))
         for i, shape in enumerate(SHAPES) for j, (xt, yt) in enumerate(TYPES)]


def _id(c):
    t = {BF16: "bf16", FP16: "fp16", FP32: "fp32", None: "8bit"}
    return "x".join(map(str, c[0])) + f"-{t[c[1]]}-{t[c[2]]}-{c[3]}-{c[4]}-{'ln' if c[5] else 'rms'}"


def _close(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got).all(), what
    bad = err > tol
    assert not bad.any(), f"{what}: off by {err[bad].max():.3g}, {float((err / tol.clamp(min=1e-300)).max()):.3g} x tolerance"


def _x(shape, xt, layout, seed):
    """(what the call takes, its values in fp64 on the CPU, dy in fp32, generator)."""
    x, dy, g = inputs(shape, seed)
    if xt is None:
        q, e = ora.pack(x.to(BF16))
        return dsv.PackedAct(q.to(torch.int8).cuda(), e.to(torch.uint8).cuda()), ora.unpack(q, e), dy, g
    x = x.to(xt)
    return lay(x.cuda(), layout), x.double(), dy, g


@pytest.mark.parametrize("case", CASES, ids=_id)
def test_norm_forward(case):
    shape, xt, yt, layout, kind, center, base = case
    x, x64, _, g = _x(shape, xt, layout, 11)
    w, b = params(kind, shape, yt, g, base)
    y, mem = guarded(shape, yt, layout)
    got, mean, rstd, kept = dsv.layer_norm_fwd(x, w.cuda() if w is not None else None, b.cuda() if b is not None else None,
                                               eps=EPS, center=center, weight_base=base, y=y, pack=xt is not None)
    assert got.data_ptr() == y.data_ptr() and outside_kept(y, mem)
    ry, rm, rr = ora.norm_fwd(x64, w, b, EPS, center, base)
    size = x64.abs().mean(-1)
    if center:
        _close(mean, rm, C * U * size, "mean")
    else:
        assert mean is None
    _close(rstd, rr, rr * (C * U + (rr * C * U * size).square()), "rstd")
    xhat = (x64 - rm[..., None]) * rr[..., None]
    gain = (w.double() + base).abs() if w is not None else torch.ones(1, dtype=torch.float64)
    shift = b.double().abs() if b is not None else 0.0
    tol = half_step(yt) * ry.abs() + C * U * gain * ((rr * size)[..., None] + xhat.abs()) + 4 * U * shift
    _close(y, ry, tol, "y")
    if xt is not None:
        q, e = ora.pack(x64)
        assert torch.equal(kept.q.cpu().long(), q) and torch.equal(kept.e.cpu().long(), e)
        again = dsv.act_pack(x)
        assert torch.equal(kept.q, again.q) and torch.equal(kept.e, again.e)


@pytest.mark.parametrize("case", CASES, ids=_id)
def test_norm_backward(case):
    shape, xt, yt, layout, kind, center, base = case
    x, x64, dy, g = _x(shape, xt, layout, 12)
    dy = dy.to(yt)
    w, b = params(kind, shape, yt, g, base)
    _, rm, rr = ora.norm_fwd(x64, None, None, EPS, center, 0.0)
    mean, rstd = (rm.float() if center else None), rr.float()
    dx, mem = guarded(shape, xt or yt, layout)
    args = (lay(dy.cuda(), LAYOUTS[(LAYOUTS.index(layout) + 1) % 4]), x, mean.cuda() if center else None, rstd.cuda(),
            w.cuda() if w is not None else None, b.cuda() if b is not None else None)
    got, dw, db = dsv.layer_norm_bwd(*args, weight_base=base, dx=dx)
    assert got.data_ptr() == dx.data_ptr() and outside_kept(dx, mem)
    rx, rw, rb = ora.norm_bwd(dy, x64, mean, rstd, w, b, base)
    xhat = (x64 - (mean.double()[..., None] if center else 0.0)) * rstd.double()[..., None]
    gg = (dy.double() * ((w.double() + base) if w is not None else 1.0)).abs()
    terms = gg + gg.mean(-1, keepdim=True) + xhat.abs() * (gg * xhat.abs()).mean(-1, keepdim=True)
    _close(dx, rx, half_step(xt or yt) * rx.abs() + C * U * rstd.double()[..., None] * terms, "dx")
    # a parameter's gradient adds at most min(rows, 1000) terms a thread and C over threads and blocks
    rows = U * (min(shape[0] * shape[1] * shape[2], 1000) + C)
    one = torch.ones(())
    for grad, ref, p, of in ((dw, rw, w, dy.double().abs() * xhat.abs()), (db, rb, b, dy.double().abs())):
        if p is None:
            assert grad is None
            continue
        assert grad.dtype == FP32 and grad.shape == p.shape
        mag = ora.norm_bwd(of, one.expand(shape), None, one.expand(shape[:-1]), None, p, 0.0)[2]
        _close(grad, ref, rows * mag, "parameter gradient")
    again = dsv.layer_norm_bwd(*args, weight_base=base, dx=guarded(shape, xt or yt, layout)[0])   # the same bits
    assert torch.equal(again[0], dx) and all(a is None or torch.equal(a, c) for a, c in zip(again[1:], (dw, db)))


#: both sides of every border between the layouts of a row over threads
WIDTHS = [7, 8, 63, 64, 65, 72, 127, 128, 129, 136, 255, 256, 257, 264, 511, 512, 513, 520, 1023, 1024, 1025, 1032, 2047,
          2048, 2049, 2056, 2561, 2568, 4095, 4096, 4097, 4104, 5120, 5121, 6152, 7167, 7176, 8184, 8185, 8191, 8192]


@pytest.mark.parametrize("xt,yt", [(BF16, BF16), (FP32, BF16), (None, BF16), (FP32, FP32)])
@pytest.mark.parametrize("D", WIDTHS)
def test_norm_of_every_width(D, xt, yt):
    """Forward, checkpoint and backward against the oracle, with more rows than a
    block takes at a time and parameters per batch."""
    shape = (2, 1, 19, D)
    x, x64, dy, g = _x(shape, xt, "bhsd", 13)
    dy = dy.to(yt)
    w, b = params("batch", shape, yt, g, 1.0)
    y, mean, rstd, kept = dsv.layer_norm_fwd(x, w.cuda(), b.cuda(), eps=EPS, weight_base=1.0, dtype=yt, pack=xt is not None)
    ry, rm, rr = ora.norm_fwd(x64, w, b, EPS, True, 1.0)
    size = x64.abs().mean(-1)
    xhat = (x64 - rm[..., None]) * rr[..., None]
    gain = (w.double() + 1.0).abs()
    _close(mean, rm, C * U * size, "mean")
    _close(rstd, rr, rr * (C * U + (rr * C * U * size).square()), "rstd")
    _close(y, ry, half_step(yt) * ry.abs() + C * U * gain * ((rr * size)[..., None] + xhat.abs()) + 4 * U * b.double().abs(), "y")
    if xt is not None:
        q, e = ora.pack(x64)
        assert torch.equal(kept.q.cpu().long(), q) and torch.equal(kept.e.cpu().long(), e)
    dx, dw, db = dsv.layer_norm_bwd(dy.cuda(), x, rm.float().cuda(), rr.float().cuda(), w.cuda(), b.cuda(), weight_base=1.0)
    rx, rw, rb = ora.norm_bwd(dy, x64, rm.float(), rr.float(), w, b, 1.0)
    xhat = (x64 - rm.float().double()[..., None]) * rr.float().double()[..., None]
    gg = (dy.double() * gain).abs()
    terms = gg + gg.mean(-1, keepdim=True) + xhat.abs() * (gg * xhat.abs()).mean(-1, keepdim=True)
    _close(dx, rx, half_step(xt or yt) * rx.abs() + C * U * rr[..., None] * terms, "dx")
    over = U * (19 + C)
    _close(dw, rw, over * (dy.double().abs() * xhat.abs()).sum(2, keepdim=True), "dweight")
    _close(db, rb, over * dy.double().abs().sum(2, keepdim=True), "dbias")


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("D", [40, 128, 517, 1024])
def test_norm_gradient_matches_differences(D, center):
    """sum dx v and sum dw u against central differences of the GPU's own
    forward in fp32. With h = 2^-6 the differences are off by h^2 / 6 times a
    third derivative (below 30 per unit of |v| |dy| here) and by the outputs'
    2^-22 / h, summed over random signs: 0.5% of the scale |dx| |v| covers both."""
    x, dy, g = inputs((1, 2, 6, D), 21, offset=0.0)
    w = torch.rand(D, generator=g) + 0.5
    v, u = torch.randn(x.shape, generator=g), torch.randn(D, generator=g)
    x, dy, w, v, u = (t.cuda() for t in (x, dy, w, v, u))
    f = lambda x, w: (dsv.layer_norm_fwd(x, w, eps=EPS, center=center)[0].double() * dy.double()).sum()  # noqa: E731
    _, mean, rstd, _ = dsv.layer_norm_fwd(x, w, eps=EPS, center=center)
    dx, dw, _ = dsv.layer_norm_bwd(dy, x, mean, rstd, w)
    h = 2.0 ** -6
    for grad, dirn, diff in ((dx, v, f(x + h * v, w) - f(x - h * v, w)), (dw, u, f(x, w + h * u) - f(x, w - h * u))):
        scale = grad.double().norm() * dirn.double().norm()
        assert abs((grad.double() * dirn.double()).sum() - diff / (2 * h)) < 5e-3 * scale


@pytest.mark.parametrize("t", [BF16, FP16, FP32])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_pack_and_unpack(shape, layout, t):
    x, _, g = inputs(shape, 31)
    x = (x * torch.exp2(torch.randint(-30 if t != FP16 else -6, 12, shape[:-1] + (1,), generator=g).float())).to(t)
    kept = dsv.act_pack(lay(x.cuda(), layout))
    q, e = ora.pack(x)
    assert torch.equal(kept.q.cpu().long(), q) and torch.equal(kept.e.cpu().long(), e)
    for out in (BF16, FP16, FP32):
        y, mem = guarded(shape, out, layout)
        assert dsv.act_unpack(kept, out=y).data_ptr() == y.data_ptr() and outside_kept(y, mem)
        assert torch.equal(y.cpu(), ora.unpack(q, e).to(out))      # one rounding, in fp16 only


def test_pack_extremes():
    """Zeros of both signs, subnormals, the largest values, ties, infinities and
    NaN; a block that is not finite leaves its neighbours alone."""
    big = torch.finfo(FP32).max
    x = torch.zeros(9, 96)
    x[0, :3] = torch.tensor([-0.0, 1e-45, -3e-42])
    x[1, :4] = torch.tensor([big, -big, big / 2, 1e30])
    x[2] = torch.arange(96) - 48 + 0.5
    x[2, ::32] = 64
    x[3, :2] = torch.tensor([float("inf"), 1.0])
    x[4, 40] = float("nan")
    x[5, 95] = float("-inf")
    x[6] = 127.5 / 64
    x[7] = torch.exp2(-torch.arange(96).float())
    x[8] = 2.0 ** -126
    for t in (FP32, BF16):
        v = x.to(t)
        kept = dsv.act_pack(v.cuda())
        q, e = ora.pack(v)
        assert torch.equal(kept.e.cpu().long(), e)
        fine = (e != 255).repeat_interleave(32, -1)
        assert torch.equal(kept.q.cpu().long()[fine], q[fine])
        back = dsv.act_unpack(kept, dtype=FP32).cpu()
        assert torch.equal(back[fine].double(), ora.unpack(q, e)[fine]) and torch.isnan(back[~fine]).all()
        assert int((~fine).sum()) == 96 + (32 if t == BF16 and not torch.isfinite(v[1]).all() else 0)


@pytest.mark.parametrize("D", [64, 128, 200, 517, 1024])
def test_rows_that_are_not_finite_stay_alone(D):
    x, dy, _ = inputs((1, 2, 33, D), 41)
    x, dy, w = x.to(BF16).cuda(), dy.to(BF16).cuda(), torch.ones(D, dtype=BF16, device="cuda")
    y0, m0, r0, _ = dsv.layer_norm_fwd(x, w)
    d0, _, _ = dsv.layer_norm_bwd(dy, x, m0, r0, w)
    hurt = x.clone()
    hurt[0, 1, 7, D // 2] = float("inf")
    hurt[0, 0, 30, 0] = float("nan")
    y, m, r, kept = dsv.layer_norm_fwd(hurt, w, pack=True)
    d, dw, _ = dsv.layer_norm_bwd(dy, hurt, m, r, w)
    d8, _, _ = dsv.layer_norm_bwd(dy, kept, m, r, w)
    rows = torch.ones(1, 2, 33, dtype=torch.bool, device="cuda")
    rows[0, 1, 7] = rows[0, 0, 30] = False
    assert torch.equal(y[rows], y0[rows]) and torch.equal(d[rows], d0[rows]) and torch.isfinite(d8[rows]).all()
    assert torch.isnan(y[~rows]).any(-1).all() and torch.isnan(d[~rows]).all() and torch.isnan(d8[~rows]).all()
    assert torch.isnan(dw).all()


@pytest.mark.parametrize("xt", [BF16, FP32])
@pytest.mark.parametrize("D", [8, 64, 80, 96, 128, 517, 1024, 5120])
def test_constant_rows(D, xt):
    """Rows of one value: nothing is left after the mean, so y is the bias, and
    neither dx (for a constant dy) nor dweight sees them; rstd is 1 / sqrt(eps)."""
    x = torch.tensor([100.0, -0.3125, 0.0, 7.25]).repeat(16)[None, :, None].expand(1, 64, D).to(xt).cuda()
    w, b = torch.rand(D, device="cuda") + 0.5, torch.randn(D, device="cuda")
    y, mean, rstd, kept = dsv.layer_norm_fwd(x, w, b, pack=True)
    assert torch.equal(y, b.to(xt).expand_as(y)) and torch.equal(mean, x[..., 0].float())
    assert ((rstd - 1e3).abs() <= 1e3 * C * U).all()
    dy = torch.ones_like(x).contiguous()
    for src in (x, kept):
        keep_x = x.float() if src is x else dsv.act_unpack(kept, dtype=FP32)
        dx, dw, db = dsv.layer_norm_bwd(dy, src, keep_x[..., 0].contiguous(), rstd, torch.ones_like(w), b)
        assert not dx.any() and not dw.any() and torch.equal(db, torch.full_like(db, 64))


@pytest.mark.parametrize("D", [64, 128, 520, 1003, 2048])
def test_rows_far_from_zero(D):
    """fp32 rows of 1000 +- 1: what the mean's own rounding costs, and no more."""
    g = torch.Generator().manual_seed(43)
    x, dy = 1000 + torch.randn(1, 2, 40, D, generator=g), torch.randn(1, 2, 40, D, generator=g)
    y, mean, rstd, _ = dsv.layer_norm_fwd(x.cuda(), eps=EPS)
    ry, rm, rr = ora.norm_fwd(x, None, None, EPS, True, 0.0)
    size = x.double().abs().mean(-1)
    _close(mean, rm, C * U * size, "mean")
    _close(y, ry, U * ry.abs() + C * U * ((rr * size)[..., None] + ry.abs()), "y")
    dx, _, _ = dsv.layer_norm_bwd(dy.cuda(), x.cuda(), mean, rstd)
    rx, _, _ = ora.norm_bwd(dy, x, mean.cpu(), rstd.cpu(), None, None, 0.0)
    gg, xh = dy.double().abs(), ((x.double() - mean.cpu().double()[..., None]) * rstd.cpu().double()[..., None]).abs()
    _close(dx, rx, U * rx.abs() + C * U * rr[..., None] * (gg + gg.mean(-1, keepdim=True) + xh * (gg * xh).mean(-1, keepdim=True)), "dx")


def test_in_place():
    for shape in ((1, 3, 70, 128), (1, 1, 5, 517), (1, 1, 4, 2048)):
        x, dy, _ = inputs(shape, 51)
        x, dy = x.to(BF16).cuda(), dy.to(BF16).cuda()
        w = torch.full(shape[-1:], 1.5, dtype=BF16, device="cuda")
        y, mean, rstd, _ = dsv.layer_norm_fwd(x, w)
        z = x.clone()
        dsv.layer_norm_fwd(z, w, y=z)
        assert torch.equal(z, y)
        dx, dw, _ = dsv.layer_norm_bwd(dy, x, mean, rstd, w)
        for which in (0, 1):
            a, b = dy.clone(), x.clone()
            got, dw2, _ = dsv.layer_norm_bwd(a, b, mean, rstd, w, dx=(a, b)[which])
            assert torch.equal(got, dx) and torch.equal(dw, dw2)


def test_repeated_input_rows():
    x, dy, _ = inputs((1, 1, 37, 128), 52)
    x, dy = x.to(BF16).cuda(), dy.to(BF16).cuda()
    wide = x.expand(3, 5, 37, 128)
    y, mean, rstd, kept = dsv.layer_norm_fwd(wide, pack=True)
    one = dsv.layer_norm_fwd(x)[0]
    assert torch.equal(y, one.expand_as(y)) and torch.equal(dsv.act_unpack(kept), dsv.act_unpack(dsv.act_pack(x)).expand_as(y))
    w = torch.ones(128, device="cuda")
    dx, _, _ = dsv.layer_norm_bwd(dy.expand_as(wide), wide, mean, rstd, w)
    assert torch.equal(dx, dx[:1, :1].expand_as(dx))


def test_no_rows():
    for shape, ps in (((0, 2, 5, 64), (64,)), ((2, 3, 0, 64), (2, 1, 1, 64)), ((2, 0, 4, 8), (2, 1, 1, 8)), ((0, 2, 4, 8), (1, 2, 1, 8)),
                      ((0, 2, 4, 8), (0, 1, 1, 8))):
        x, w = torch.empty(shape, dtype=BF16, device="cuda"), torch.ones(ps, device="cuda")
        y, mean, rstd, kept = dsv.layer_norm_fwd(x, w, w, pack=True)
        assert y.shape == shape and rstd.shape == shape[:-1]
        for src in (x, kept):
            dx, dw, db = dsv.layer_norm_bwd(x, src, mean, rstd, w, w)
            assert dx.shape == shape and (dw == 0).all() and (db == 0).all() and dw.shape == ps
        assert dsv.act_unpack(dsv.act_pack(x)).shape == shape


def test_modulation_slices():
    """Shift and scale as slices of one [B, 6 D] projection: rows of parameters with a stride."""
    B, S, D = 3, 50, 256
    x, dy, g = inputs((B, 1, S, D), 61)
    mod = (0.3 * torch.randn(B, 6 * D, generator=g)).to(BF16)
    x, dy = x.to(BF16).squeeze(1).cuda(), dy.to(BF16).squeeze(1).cuda()
    shift, scale = (t[:, None] for t in mod.cuda().chunk(6, -1)[2:4])
    y, mean, rstd, _ = dsv.layer_norm_fwd(x, scale, shift, weight_base=1.0)
    dx, dw, db = dsv.layer_norm_bwd(dy, x, mean, rstd, scale, shift, weight_base=1.0)
    y2, _, _, _ = dsv.layer_norm_fwd(x, scale.contiguous(), shift.contiguous(), weight_base=1.0)
    ref = ora.norm_bwd(dy.cpu(), x.cpu(), mean.cpu(), rstd.cpu(), scale.cpu(), shift.cpu(), 1.0)
    assert torch.equal(y, y2) and dw.shape == (B, 1, D)
    for a, r in zip((dw, db), ref[1:]):
        assert (a.double().cpu() - r).norm() < 1e-6 * r.norm()


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements apart, in the input, the output and the gradient."""
    far = (1 << 31) + 8 * 1024
    mem = torch.empty(far + 4096, dtype=BF16, device="cuda")
    x, dy, _ = inputs((2, 1, 3, 128), 71)
    x, dy, w = x.to(BF16).cuda(), dy.to(BF16).cuda(), torch.ones(2, 1, 1, 128, device="cuda")
    at = lambda shift: mem[shift:].as_strided((2, 1, 3, 128), (far, far, 128, 1))  # noqa: E731
    xf, yf = at(0), at(1024)
    xf.copy_(x)
    y, mean, rstd, kept = dsv.layer_norm_fwd(xf, w, y=yf, pack=True)
    ref, m, r, k = dsv.layer_norm_fwd(x, w, pack=True)
    assert torch.equal(y, ref) and torch.equal(kept.q, k.q) and torch.equal(rstd, r)
    dx, dw, _ = dsv.layer_norm_bwd(dy, xf, mean, rstd, w, dx=at(2048))
    rx, rw, _ = dsv.layer_norm_bwd(dy, x, m, r, w)
    assert torch.equal(dx, rx) and torch.equal(dw, rw)
    assert torch.equal(dsv.act_unpack(kept, out=at(2048)), dsv.act_unpack(k))
    assert torch.equal(dsv.act_pack(at(2048)).q, dsv.act_pack(dsv.act_unpack(k)).q)


@pytest.mark.parametrize("shape,ps", [((20, 24, 200, 64), (20, 24, 1, 64)), ((700, 1, 37, 128), (700, 1, 1, 128)),
                                      ((1, 400, 90, 517), (1, 400, 1, 517)), ((2, 300, 20, 1032), (1, 300, 1, 1032)),
                                      ((300, 1, 3, 5120), (300, 1, 1, 5120))])
def test_more_groups_than_blocks(shape, ps):
    """Hundreds of parameter rows, some of whose rows fall to two blocks. Against
    fp64 sums on the GPU; U (rows + C) covers a thread's additions and the joins."""
    g = torch.Generator(device="cuda").manual_seed(73)
    x = torch.randn(shape, device="cuda", generator=g).to(BF16)
    dy = torch.randn(shape, device="cuda", generator=g).to(BF16)
    w, b = torch.rand(ps, device="cuda", generator=g) + 0.5, torch.randn(ps, device="cuda", generator=g)
    y, mean, rstd, kept = dsv.layer_norm_fwd(x, w, b, pack=True)
    xhat = (x.double() - mean.double()[..., None]) * rstd.double()[..., None]
    ref = xhat * w.double() + b.double()
    assert ((y.double() - ref).abs() <= half_step(BF16) * ref.abs() + C * U * (xhat.abs() + 3) * 3).all()
    dims = [i for i in range(3) if ps[i] == 1]
    rows = 1
    for i in dims:
        rows *= shape[i]
    for src, xh in ((x, xhat), (kept, (dsv.act_unpack(kept).double() - mean.double()[..., None]) * rstd.double()[..., None])):
        dx, dw, db = dsv.layer_norm_bwd(dy, src, mean, rstd, w, b)
        for grad, term in ((dw, dy.double() * xh), (db, dy.double())):
            err = (grad.double() - term.sum(dims, keepdim=True)).abs()
            assert (err <= U * (rows + C) * term.abs().sum(dims, keepdim=True)).all()
        again = dsv.layer_norm_bwd(dy, src, mean, rstd, w, b)
        assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))


def test_more_than_2_31_channels():
    """An activation of 2^32 channels: its last rows are those of a small call."""
    x = torch.empty(1, 16, 262144, 1024, dtype=BF16, device="cuda").normal_()
    w = torch.rand(1024, device="cuda") + 0.5
    y, mean, rstd, kept = dsv.layer_norm_fwd(x, w, pack=True)
    tail = x[:, 15:, -70:]
    ty, tm, tr, tk = dsv.layer_norm_fwd(tail, w, pack=True)
    assert torch.equal(y[:, 15:, -70:], ty) and torch.equal(mean[:, 15:, -70:], tm) and torch.equal(rstd[:, 15:, -70:], tr)
    assert torch.equal(kept.q[:, 15:, -70:], tk.q) and torch.equal(kept.e[:, 15:, -70:], tk.e)
    back = dsv.act_unpack(kept, out=y)
    assert torch.equal(back[:, 15:, -70:], dsv.act_unpack(tk))
    dx, dw, _ = dsv.layer_norm_bwd(x, kept, mean, rstd, w, dx=y)
    tdx, _, _ = dsv.layer_norm_bwd(tail, tk, tm, tr, w)
    assert torch.equal(dx[:, 15:, -70:], tdx) and torch.isfinite(dw).all()


@pytest.mark.parametrize("shape", [(1, 4, 3000, 64), (1, 1, 700, 517), (2, 1, 900, 1024)])
def test_calls_in_a_row_on_the_same_memory(shape):
    """Kernels that overlap in their launches still run one after the other: calls
    that overwrite each other's inputs give the same with and without a wait
    between them."""
    x0, dy0, _ = inputs(shape, 97)
    x0, dy0 = x0.to(BF16).cuda(), dy0.to(BF16).cuda()
    w = torch.rand(shape[-1], device="cuda") + 0.5
    ws = torch.empty(max(dsv.layer_norm_bwd_workspace_size(x0, w), 256), dtype=torch.uint8, device="cuda")

    def run(wait):
        x, dy, kept, out = x0.clone(), dy0.clone(), dsv.act_pack(dy0), []
        for i in range(30):
            _, mean, rstd, _ = dsv.layer_norm_fwd(x, w, y=x, pack=kept)
            wait()
            dsv.act_unpack(kept, out=x)
            wait()
            _, dw, _ = dsv.layer_norm_bwd(dy, kept, mean, rstd, w, dx=dy, workspace=ws)
            wait()
            dsv.act_pack(dy, out=kept)
            wait()
            dsv.act_unpack(kept, out=dy)
            wait()
            x.add_(dy)
            out.append(dw)
        return [x, dy, kept.q, kept.e] + out

    a, b = run(lambda: None), run(torch.cuda.synchronize)
    assert torch.isfinite(a[0]).all() and all(torch.equal(p, q) for p, q in zip(a, b))


def test_calls_at_once():
    """Calls on two streams, each with its own outputs, give what they give alone."""
    ins = []
    for i in range(2):
        x, dy, _ = inputs((1, 6, 20000, 128), 91 + i)
        ins.append((x.to(BF16).cuda(), dy.to(BF16).cuda(), torch.rand(128, device="cuda") + 0.5))

    def step(x, dy, w):
        y, mean, rstd, kept = dsv.layer_norm_fwd(x, w, pack=True)
        return (y, kept.q, kept.e, dsv.act_unpack(kept)) + dsv.layer_norm_bwd(dy, kept, mean, rstd, w, w)

    alone = [step(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    for _ in range(5):
        outs = []
        for s, i in zip(streams, ins):
            with torch.cuda.stream(s):
                outs.append(step(*i))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for a, o in zip(alone, outs) for p, q in zip(a, o))


def test_graphs_and_streams():
    """Captured once, replayed on new inputs; two graphs that share a workspace,
    replayed in turn on one stream; calls on a stream of the caller's."""
    shape = (1, 4, 3000, 128)
    x, dy, _ = inputs(shape, 81)
    x, dy, w = x.to(BF16).cuda(), dy.to(BF16).cuda(), torch.rand(128, device="cuda") + 0.5
    ws = torch.empty(dsv.layer_norm_bwd_workspace_size(x, w), dtype=torch.uint8, device="cuda")

    def step():
        y, mean, rstd, kept = dsv.layer_norm_fwd(x, w, pack=True)
        return (y, kept.q, kept.e) + dsv.layer_norm_bwd(dy, kept, mean, rstd, w, w, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, first))
    x.mul_(-2)
    dy.mul_(0.5)
    ref = [t.clone() for t in step()]
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_small_workspace_is_refused():
    x = torch.zeros(1, 4, 3000, 128, dtype=BF16, device="cuda")
    r = torch.ones(1, 4, 3000, device="cuda")
    w = torch.ones(128, device="cuda")
    need = dsv.layer_norm_bwd_workspace_size(x, w)
    with pytest.raises(ValueError):
        dsv.layer_norm_bwd(x, x, None, r, w, workspace=torch.empty(need - 256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        dsv.layer_norm_bwd(x, x, None, r, w, workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(dsv.DsvError) as err:
        dsv.layer_norm_bwd(x, x, None, r, w, workspace=torch.empty(need + 8, dtype=torch.uint8, device="cuda")[8:])
    assert err.value.code == 3


def test_parameter_layouts():
    """Which rows share parameters, by the parameter's shape; anything else is refused."""
    shape = (2, 3, 5, 8)
    x = torch.randn(shape, device="cuda")
    z = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    ref = dsv.layer_norm_fwd(x)[0]
    _, mean, rstd, _ = dsv.layer_norm_fwd(x)
    for p in (z(8), z(1, 1, 1, 8), z(2, 1, 1, 8), z(1, 3, 1, 8), z(2, 3, 1, 8), z(2, 48).view(2, 1, 6, 8)[:, :, 2:3]):
        assert torch.equal(dsv.layer_norm_fwd(x, p)[0], ref)
        assert dsv.layer_norm_bwd(x, x, mean, rstd, p)[1].shape == p.shape
    for p in (z(3, 1, 8), z(1, 1, 8), z(8)):
        assert torch.equal(dsv.layer_norm_fwd(x[0], p)[0], ref[0])
    assert torch.equal(dsv.layer_norm_fwd(x[0, 0], z(1, 8))[0], ref[0, 0])
    for bad in (z(7), z(2, 8), z(5, 8), z(2, 1, 5, 8), z(3, 1, 1, 8), z(16)[::2], z(2, 3, 8), z(()), z(8).to(torch.int32),
                z(8).cpu(), z(8).double()):
        for call in (lambda: dsv.layer_norm_fwd(x, bad), lambda: dsv.layer_norm_fwd(x, None, bad),
                     lambda: dsv.layer_norm_bwd(x, x, mean, rstd, bad)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        dsv.layer_norm_fwd(x, z(8), z(8).to(BF16))
    with pytest.raises(ValueError):
        dsv.layer_norm_fwd(x, z(8), z(1, 1, 1, 8))


def test_refused_tensors():
    x = torch.randn(2, 3, 5, 8, device="cuda")
    y, mean, rstd, kept = dsv.layer_norm_fwd(x, pack=True)
    for call in (lambda: dsv.layer_norm_fwd(x.transpose(2, 3)), lambda: dsv.layer_norm_fwd(x.int()),
                 lambda: dsv.layer_norm_fwd(x, y=y[:1]), lambda: dsv.layer_norm_fwd(x, y=y, dtype=BF16),
                 lambda: dsv.layer_norm_fwd(x, dtype=torch.int8), lambda: dsv.layer_norm_fwd(x[0, 0, 0]),
                 lambda: dsv.layer_norm_fwd(x[None]), lambda: dsv.layer_norm_fwd(x, pack=dsv.PackedAct(kept.q[:1], kept.e)),
                 lambda: dsv.layer_norm_bwd(y, x, mean, rstd.double()), lambda: dsv.layer_norm_bwd(y, x, mean[:1], rstd),
                 lambda: dsv.layer_norm_bwd(y, x, mean, None), lambda: dsv.layer_norm_bwd(y.cpu(), x, mean, rstd),
                 lambda: dsv.layer_norm_bwd(y, dsv.PackedAct(kept.q, kept.e[..., :0]), mean, rstd),
                 lambda: dsv.act_pack(kept), lambda: dsv.act_pack(x, out=(kept.q, kept.e)), lambda: dsv.act_unpack(x),
                 lambda: dsv.act_unpack(dsv.PackedAct(kept.q.float(), kept.e)), lambda: dsv.act_unpack(kept, out=y.cpu()),
                 lambda: dsv.act_unpack(kept, dtype=torch.float64), lambda: dsv.act_unpack(kept, dtype="bf16")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: dsv.layer_norm_fwd(x, eps=0.0), lambda: dsv.layer_norm_fwd(x, y=x.expand(2, 3, 5, 8)[:, :, :1].expand_as(x)),
                 lambda: dsv.layer_norm_fwd(x.to(BF16), dtype=FP32), lambda: dsv.layer_norm_bwd(y.to(BF16), x.to(FP16), mean, rstd)):
        with pytest.raises(dsv.DsvError):
            call()

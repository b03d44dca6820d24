"""The fp64 oracle of the row calls, pinned by differences, by torch's own
autograd and by hand-made blocks (CPU)."""
import pytest
import torch

from oracle import rows_oracle as ora


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("pshape", [(6,), (2, 1, 1, 6), (1, 3, 1, 6)])
def test_norm_gradients_match_differences(center, pshape):
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, dy, w, b, base, eps = rn(2, 3, 4, 6), rn(2, 3, 4, 6), rn(*pshape), rn(*pshape), 1.0, 1e-6
    _, mean, rstd = ora.norm_fwd(x, w, b, eps, center, base)
    got = ora.norm_bwd(dy, x, mean if center else None, rstd, w, b, base)
    loss = lambda x, w, b: (dy * ora.norm_fwd(x, w, b, eps, center, base)[0]).sum()  # noqa: E731
    h = 1e-6
    for which, (at, grad) in enumerate(zip((x, w, b), got)):
        for i in range(at.numel()):
            up, down = at.clone(), at.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            args = [[x, w, b], [x, w, b]]
            args[0][which], args[1][which] = up, down
            # central differences: error ~ h^2 + 2^-53 |loss| / h < 1e-8
            assert abs((loss(*args[0]) - loss(*args[1])) / (2 * h) - grad.reshape(-1)[i]) < 1e-6


@pytest.mark.parametrize("center", [True, False])
def test_norm_matches_autograd(center):
    g = torch.Generator().manual_seed(4)
    x = torch.randn(3, 5, 7, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(7, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(3, 5, 7, generator=g, dtype=torch.float64)
    y, mean, rstd = ora.norm_fwd(x, w, None, 1e-5, center, 0.0)
    y.backward(dy)
    dx, dw, _ = ora.norm_bwd(dy, x.detach(), mean.detach() if center else None, rstd.detach(), w.detach(), None, 0.0)
    torch.testing.assert_close(dx, x.grad, rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(dw, w.grad, rtol=1e-12, atol=1e-12)


def test_pack_by_hand():
    x = torch.zeros(1, 40)
    x[0, :5] = torch.tensor([1.0, -0.5, 127.5 / 64, 1.5 / 64, 2.5 / 64])   # top 1.99..: step 2^-6
    x[0, 32] = 3e38
    q, e = ora.pack(x)
    assert e.tolist() == [[127, 254]]
    assert q[0, :5].tolist() == [64, -32, 127, 2, 2]        # ties to even, 127.5 -> 128 -> 127
    assert q[0, 32] == 113 and torch.isfinite(ora.unpack(q, e)).all()


def test_pack_of_nothing_and_not_finite():
    q, e = ora.pack(torch.zeros(2, 33))
    assert (q == 0).all() and (e == 7).all()
    x = torch.ones(1, 64)
    x[0, 3], x[0, 4] = float("inf"), float("nan")
    r = ora.unpack(*ora.pack(x))
    assert torch.isnan(r[0, :32]).all() and (r[0, 32:] == 1).all()


def test_pack_error_is_half_a_step():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(50, 96, generator=g) * torch.exp(4 * torch.randn(50, 1, generator=g))
    q, e = ora.pack(x)
    step = torch.exp2(e.double() - 133).repeat_interleave(32, -1)
    top = x.double().abs() > 127.5 * step
    err = (ora.unpack(q, e) - x.double()).abs() / step
    assert err[~top].max() <= 0.5 and err.max() <= 1.0
    r = ora.unpack(q, e)
    assert torch.equal(r, r.to(torch.bfloat16).double())     # exact in bf16
    q2, e2 = ora.pack(r)
    assert torch.equal(q2[e2.repeat_interleave(32, -1) == e.repeat_interleave(32, -1)],
                       q[e2.repeat_interleave(32, -1) == e.repeat_interleave(32, -1)])

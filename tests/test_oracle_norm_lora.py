"""Pins of the 64-bit layer-norm and adapter oracle (CPU): torch's autograd in
float64, central differences and closed forms, none of which share its code."""
import numpy as np
import pytest
import torch

from oracle import norm_lora as o


def _t(g, *shape):
    return torch.randn(shape, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_against_autograd(affine):
    g = torch.Generator().manual_seed(3)
    x, dy = _t(g, 5, 48).requires_grad_(), _t(g, 5, 48)
    ga, be = _t(g, 48).requires_grad_(), _t(g, 48).requires_grad_()
    want = torch.nn.functional.layer_norm(x, (48,), ga if affine else None, be if affine else None, 1e-5)
    want.backward(dy)
    y, mean, rstd = o.layer_norm_forward(x.detach(), ga.detach() if affine else None, be.detach() if affine else None, 1e-5)
    assert np.allclose(y, want.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dg, db = o.layer_norm_backward(dy, x.detach(), mean, rstd, ga.detach() if affine else None)
    assert np.allclose(dx, x.grad.numpy(), rtol=1e-11, atol=1e-12)
    if affine:
        assert np.allclose(dg, ga.grad.numpy(), rtol=1e-12, atol=1e-12)
        assert np.allclose(db, be.grad.numpy(), rtol=1e-12, atol=1e-12)


def test_layer_norm_closed_form():
    # one +c and one -c in a row of zeros: mean 0, var 2 c^2 / K
    x = torch.zeros((1, 32), dtype=torch.float64)
    x[0, 3], x[0, 9] = 4.0, -4.0
    y, mean, rstd = o.layer_norm_forward(x, eps=0.0)
    assert mean[0] == 0.0 and abs(rstd[0] - 1.0) < 1e-15
    assert np.array_equal(y, x.numpy())


def _lora_case(seed):
    g = torch.Generator().manual_seed(seed)
    M, K, N, L, R = 7, 16, 9, 3, 8
    idx = np.array([2, 0, -1, 2, 5, 0, 2])   # adapter 1 has no rows, rows 2 and 4 have no adapter
    return (_t(g, M, K), _t(g, L, R, K), _t(g, L, N, R), torch.rand(L, generator=g, dtype=torch.float64) + 0.5, idx, _t(g, M, N),
            _t(g, M, N), _t(g, M, K))


def test_lora_against_autograd():
    x, A, B, s, idx, y0, dy, dx0 = _lora_case(1)
    x, A, B = x.requires_grad_(), A.requires_grad_(), B.requires_grad_()
    on = torch.tensor([(0 <= i < 3) for i in idx], dtype=torch.float64)
    safe = torch.tensor([i if 0 <= i < 3 else 0 for i in idx])
    h = torch.einsum("mk,mrk->mr", x, A[safe])
    want = y0 + on[:, None] * s[safe][:, None] * torch.einsum("mr,mnr->mn", h, B[safe])
    want.backward(dy)
    y, h64 = o.lora_forward(x.detach(), A.detach(), B.detach(), s, idx, y0)
    assert np.allclose(y, want.detach().numpy(), rtol=1e-12, atol=1e-12)
    assert np.isnan(h64[[2, 4]]).all() and np.isfinite(h64[[0, 1, 3, 5, 6]]).all()
    dx, dA, dB, _ = o.lora_backward(dy, x.detach(), A.detach(), B.detach(), s, idx, np.nan_to_num(h64), dx0)
    assert np.allclose(dx - dx0.numpy(), x.grad.numpy(), rtol=1e-11, atol=1e-12)
    assert np.allclose(dA, A.grad.numpy(), rtol=1e-11, atol=1e-12) and np.all(dA[1] == 0)
    assert np.allclose(dB, B.grad.numpy(), rtol=1e-11, atol=1e-12) and np.all(dB[1] == 0)


def test_gradients_against_differences():
    # <dY, f(x + e d) - f(x - e d)> / 2e against the oracle's gradients, along one random direction each
    x, A, B, s, idx, y0, dy, _ = _lora_case(2)
    g = torch.Generator().manual_seed(9)
    e = 1e-5
    _, h = o.lora_forward(x, A, B, s, idx, y0)
    dx, dA, dB, _ = o.lora_backward(dy, x, A, B, s, idx, np.nan_to_num(h), torch.zeros_like(x))
    for grad, args in ((dx, 0), (dA, 1), (dB, 2)):
        v = [x, A, B]
        d = _t(g, *v[args].shape)
        lo, hi = list(v), list(v)
        lo[args], hi[args] = v[args] - e * d, v[args] + e * d
        num = ((o.lora_forward(*hi, s, idx, y0)[0] - o.lora_forward(*lo, s, idx, y0)[0]) * dy.numpy()).sum() / (2 * e)
        assert abs(num - (grad * d.numpy()).sum()) <= 1e-7 * max(1.0, abs(num))
    xn, gamma, dyn = _t(g, 4, 16), _t(g, 16), _t(g, 4, 16)
    _, mean, rstd = o.layer_norm_forward(xn, gamma, eps=1e-6)
    dxn, dgn, _ = o.layer_norm_backward(dyn, xn, mean, rstd, gamma)
    d = _t(g, 4, 16)
    num = ((o.layer_norm_forward(xn + e * d, gamma)[0] - o.layer_norm_forward(xn - e * d, gamma)[0]) * dyn.numpy()).sum() / (2 * e)
    assert abs(num - (dxn * d.numpy()).sum()) <= 1e-7 * max(1.0, abs(num))
    d = _t(g, 16)
    num = ((o.layer_norm_forward(xn, gamma + e * d)[0] - o.layer_norm_forward(xn, gamma - e * d)[0]) * dyn.numpy()).sum() / (2 * e)
    assert abs(num - (dgn * d.numpy()).sum()) <= 1e-7 * max(1.0, abs(num))

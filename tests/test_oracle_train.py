"""The oracle of the layer norm, the two-level products and the weight update
against float64 torch operators, autograd, differences and closed forms (CPU)."""
import numpy as np
import pytest
import torch

from oracle import train


@pytest.mark.parametrize("shape", [(1, 1, 1, 1), (2, 3, 4, 5), (1, 1, 7, 64), (3, 1, 2, 33)])
def test_layer_norm_is_torchs(shape):
    rng = np.random.default_rng(sum(shape))
    x, dy, skip = (rng.standard_normal(shape) for _ in range(3))
    c = shape[-1]
    gamma, beta = rng.standard_normal(c), rng.standard_normal(c)
    t = [torch.from_numpy(v).requires_grad_() for v in (x, gamma, beta)]
    y = torch.nn.functional.layer_norm(t[0], (c,), t[1], t[2], 1e-5)
    got, mean, rstd = train.layer_norm(x, gamma, beta, 1e-5)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=0, atol=1e-12 * max(1, np.abs(got).max()))
    # the loss also takes x itself, as a skip path does
    ((y * torch.from_numpy(dy)).sum() + (t[0] * torch.from_numpy(skip)).sum()).backward()
    dx, dgamma, dbeta, _ = train.layer_norm_backward(dy, x, gamma, mean, rstd, skip)
    scale = 1 + np.abs(rstd).max()
    for a, b in ((dx, t[0].grad), (dgamma, t[1].grad), (dbeta, t[2].grad)):
        np.testing.assert_allclose(a, b.numpy(), rtol=0, atol=1e-11 * scale * max(1, np.abs(a).max()))


def test_layer_norm_gradient_by_differences():
    rng = np.random.default_rng(3)
    shape = (2, 2, 3, 19)
    x, dy, v = (rng.standard_normal(shape) for _ in range(3))
    gamma, beta = rng.standard_normal(19), rng.standard_normal(19)
    _, mean, rstd = train.layer_norm(x, gamma, beta, 1e-5)
    dx = train.layer_norm_backward(dy, x, gamma, mean, rstd)[0]
    f = lambda s: (train.layer_norm(x + s * v, gamma, beta, 1e-5)[0] * dy).sum()  # noqa: E731
    assert abs((f(1e-4) - f(-1e-4)) / 2e-4 - (dx * v).sum()) <= 1e-6 * np.abs(dx * v).sum()


NEWTON = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("shape", [(1, 1), (5, 5), (7, 20), (20, 7), (16, 33)])
def test_newton_steps_act_on_the_singular_values_alone(shape):
    rng = np.random.default_rng(shape[0])
    g = rng.standard_normal(shape)
    u, s, v = np.linalg.svd(g, full_matrices=False)
    s = s / (np.linalg.norm(g) + 1e-7)
    a, b, c = NEWTON
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    np.testing.assert_allclose(train.newton(g, 5, a, b, c, 1e-7), (u * s) @ v, rtol=0, atol=1e-11)
    # cubic steps towards the polar factor
    np.testing.assert_allclose(train.newton(g, 32, 1.5, -0.5, 0.0, 0.0), u @ v, rtol=0, atol=1e-9)


def test_muon_step_by_hand():
    # one row: X(U) = p^5(1) U / |U|
    g, m, w = np.array([[3.0, 4.0]]), np.array([[0.0, 1.0]]), np.array([[1.0, -1.0]])
    p = 1.0
    for _ in range(5):
        p = 3.4445 * p - 4.7750 * p ** 3 + 2.0315 * p ** 5
    m2, w2 = train.muon(g, m, w, 0.1, 0.5, 0.2, False, 0, (5, *NEWTON, 0.0))
    np.testing.assert_allclose(m2, [[3.0, 4.5]], rtol=1e-15)
    np.testing.assert_allclose(w2, 0.98 * w - 0.1 * p * m2 / np.hypot(3, 4.5), rtol=1e-13)
    _, w3 = train.muon(g.T, m.T, w.T, 0.1, 0.5, 0.2, True, 1, (5, *NEWTON, 0.0))
    u = g + 0.5 * m2
    np.testing.assert_allclose(w3.T, 0.98 * w - 0.1 * np.sqrt(2) * p * u / np.linalg.norm(u), rtol=1e-13)
    _, w4 = train.muon(g, m, w, 0.1, 0.5, 0.0, True, 2, (5, *NEWTON, 0.0))
    np.testing.assert_allclose(w4, w - 0.1 * 0.2 * np.sqrt(2) * p * u / np.linalg.norm(u), rtol=1e-13)

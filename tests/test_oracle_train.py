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

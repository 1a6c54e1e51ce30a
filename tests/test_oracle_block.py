"""Pins of the fp64 oracle of group norm, dropout and the replay cache
(oracle/block.py) that do not rest on it: torch's float64 group norm and
autograd, differences, the published Philox vectors, hand-worked values."""
import numpy as np
import pytest
import torch

import oracle
from oracle import block

TORCH_ACT = [lambda u: u, torch.relu, torch.nn.functional.silu, torch.nn.functional.gelu]


def _case(seed, shape, groups):
    rng = np.random.default_rng(seed)
    c = shape[-1]
    return (rng.standard_normal(shape) * 1.7 + 0.4, rng.standard_normal(shape), 1 + 0.2 * rng.standard_normal(c),
            0.3 * rng.standard_normal(c))


@pytest.mark.parametrize("kind", range(4))
@pytest.mark.parametrize("shape,groups", [((3, 4, 2, 12), 3), ((1, 5, 3, 7), 7), ((2, 2, 1, 10), 1)])
def test_group_norm_against_torch_float64(kind, shape, groups):
    x, dy, gamma, beta = _case(kind, shape, groups)
    rng = np.random.default_rng(9)
    factor = np.where(rng.random(shape) < 0.3, 0.0, 1 / 0.7)
    t = lambda a: torch.tensor(a, requires_grad=True)  # noqa: E731
    tx, tg, tb = t(x), t(gamma), t(beta)
    y = TORCH_ACT[kind](torch.nn.functional.group_norm(tx.permute(2, 3, 0, 1), groups, tg, tb, 1e-3))
    y = y.permute(2, 3, 0, 1) * torch.tensor(factor)
    y.backward(torch.tensor(dy))
    oy, mean, rstd, _ = block.group_norm(x, gamma, beta, groups, kind, 1e-3, factor)
    np.testing.assert_allclose(oy, y.detach().numpy(), rtol=1e-11, atol=1e-12)
    dx, dgamma, dbeta, _ = block.group_norm_backward(dy, x, gamma, beta, mean, rstd, groups, kind, factor)
    np.testing.assert_allclose(dx, tx.grad.numpy(), rtol=1e-9, atol=1e-11)
    np.testing.assert_allclose(dgamma, tg.grad.numpy(), rtol=1e-9, atol=1e-11)
    np.testing.assert_allclose(dbeta, tb.grad.numpy(), rtol=1e-9, atol=1e-11)


def test_group_norm_gradient_against_differences():
    shape, groups = (3, 2, 2, 6), 2
    for kind in (block.ACT_NONE, block.ACT_SILU, block.ACT_GELU):
        x, dy, gamma, beta = _case(20 + kind, shape, groups)
        _, mean, rstd, _ = block.group_norm(x, gamma, beta, groups, kind, 1e-5)
        dx, dgamma, dbeta, _ = block.group_norm_backward(dy, x, gamma, beta, mean, rstd, groups, kind)
        rng = np.random.default_rng(3)
        v, vg, vb = rng.standard_normal(shape), rng.standard_normal(6), rng.standard_normal(6)
        h = 1e-5
        f = lambda s: (block.group_norm(x + s * v, gamma + s * vg, beta + s * vb, groups, kind, 1e-5)[0] * dy).sum()  # noqa: E731
        assert (f(h) - f(-h)) / (2 * h) == pytest.approx((dx * v).sum() + dgamma @ vg + dbeta @ vb, rel=1e-7)


def test_philox_words_are_the_known_generator():
    words = block.philox_words(5, 3, 0x0123456789ABCDEF)
    for row in range(5):
        for o in range(3):
            ref = oracle.philox4x32_10((row, o, 1, 0), (0x89ABCDEF, 0x01234567))
            assert list(words[row, o]) == [int(v) for v in ref]


def test_drop_factor_rate_and_edges():
    f = block.drop_factor((40, 50, 4, 37), 0.25, 77)
    assert set(np.unique(f)) == {0.0, float(np.float32(65536 / 49152))}
    assert abs((f == 0).mean() - 0.25) < 4 * np.sqrt(0.25 * 0.75 / f.size)
    assert (block.drop_factor((2, 2, 2, 9), 0.0, 1) == 1).all()
    assert (block.drop_factor((2, 2, 2, 9), 1.0, 1) == 0).all()
    assert (block.drop_factor((2, 2, 2, 9), 1e-6, 1) == 1).all()  # rounds to no dropping at all
    a, b = block.drop_factor((8, 8, 2, 32), 0.5, 1), block.drop_factor((8, 8, 2, 32), 0.5, 2)
    assert (a != b).any()
    # a row's numbers do not depend on how many rows there are
    assert (block.drop_factor((1, 1, 3, 20), 0.5, 5) == block.drop_factor((1, 1, 9, 20), 0.5, 5)[:, :, :3]).all()


@pytest.mark.parametrize("fmt", range(5))
def test_cache_lines_are_each_samples_own_quantization(fmt):
    rng = np.random.default_rng(fmt)
    x = rng.standard_normal((3, 2, 4, 45))
    codes, scales = block.cache_lines(x, fmt)
    c, s, _ = oracle.quantize(oracle.ROLE_ACT, fmt, 1, x)  # lines do not see the other samples
    ref = oracle.pack(fmt, c).reshape(3, 2, 4, -1)
    np.testing.assert_array_equal(codes.reshape(4, 3, 2, -1), ref.transpose(2, 0, 1, 3))
    np.testing.assert_array_equal(scales.reshape(4, 3, 2, -1), s.reshape(3, 2, 4, -1).transpose(2, 0, 1, 3))
    v = block.cache_values(codes, scales, fmt, 3, 2, 45)
    np.testing.assert_array_equal(v, oracle.dequantize(oracle.ROLE_ACT, fmt, 1, c, s))
    # storing what was read changes nothing
    c2, s2 = block.cache_lines(v, fmt)
    np.testing.assert_array_equal(c2, codes)
    np.testing.assert_array_equal(s2, scales)

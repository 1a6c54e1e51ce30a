"""The orthogonalised weight update of full calls: 32 weights of every size of
tile share the launches, each with the result of a call of its own, bit for bit. Very long rows."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
from gpu_common import dev, host, say, workspace
from test_gpu_update import E, MUON, SHAPES, _gradient, _one_step_bound, _run, f32

pytestmark = pytest.mark.gpu

# large matrices (tiles of 256 x 128 with slices) first, last, side by side and between small ones, tall and wide
GROUP = [(1550, 2600), *SHAPES[:9], (1800, 1800), (2100, 1100), *SHAPES[9:], (700, 700), (512, 2048), (48, 7000), (256, 1152),
         (768, 500), (3, 5), (1, 1), (1100, 2050), (1024, 1024), (1536, 640)][:31] + [(2048, 1300)]


def test_full_calls_of_all_sizes():
    assert len(GROUP) == mq.UPDATE_GROUP_MAX
    mats = [_gradient(s, 200 + k) for k, s in enumerate(GROUP)]
    nt = mq.mq_newton(2)
    got = _run(nt, mats)
    for g, x in zip(mats, got):
        say(f"{g.shape}")
        np.testing.assert_array_equal(_run(nt, [g], fill=0)[0], x)
    for order in (range(31, -1, -1), [*range(16, 32), *range(16)]):
        for k, x in zip(order, _run(nt, [mats[k] for k in order])):
            np.testing.assert_array_equal(x, got[k])


def test_a_full_optimizer_step():
    g, m, w = ([dev(_gradient(s, 300 + 50 * j + k)) for k, s in enumerate(GROUP)] for j in range(3))
    opt = mq.mq_muon(0.02, 0.95, 0.01, True, mq.MUON_SCALE_ASPECT, newton=mq.mq_newton(2))
    alone = [[t.clone() for t in v] for v in (m, w)]
    ws = workspace(mq.mqconv_orthogonalize_workspace_bytes(GROUP)).fill_(0xFF)
    mq.mqconv_muon_update(opt, g, m, w, ws)
    for k, s in enumerate(GROUP):
        say(f"{s}")
        mq.mqconv_muon_update(opt, g[k:k + 1], alone[0][k:k + 1], alone[1][k:k + 1], ws)
        assert torch.equal(m[k], alone[0][k]) and torch.equal(w[k], alone[1][k])
        assert np.isfinite(host(w[k])).all()


@pytest.mark.parametrize("shape", [(1, 2 ** 20 + 5), (3, 300001), (300001, 2), (40, 70003)], ids=str)
def test_very_long_rows(shape):
    """A step is held to the bound of test_gpu_update.py element by element, which grows with the number n of a sum's terms, and
    in the 2-norm to what roundings of either sign add up to: S is summed in 32 slices at the most, 16 products at a time, so
    n / 512 roundings of 2^-24 of it and more, 4 e sqrt(n / 512) with four deviations; F = a + b S + c S^2 takes that times
    (|b| x^2 + 2 |c| x^4) / F <= 12.7 (at x = 1, F = 0.70). 2^-16 + 2^-18 is for
    the parts of X, S and F, 38 of 2^-22 there and less elsewhere, with what X and X1 are rounded by."""
    coef = tuple(f32(v) for v in MUON)
    g = _gradient(shape, 77, "noise")
    got = _run(mq.mq_newton(1, *coef, 1e-7), [g])[0]
    ref, tol = _one_step_bound(g, *coef, f32(1e-7))
    say(f"{shape}: {np.abs(got - ref).max():.2e}, of the bound {np.max(np.abs(got - ref) / tol):.2f}")
    assert (np.abs(got - ref) <= 1.01 * tol).all()
    assert np.linalg.norm(got - ref) <= (2.0 ** -18 + 2.0 ** -16 + 12.7 * 4 * E * np.sqrt(max(shape) / 512)) * np.linalg.norm(ref)

"""Group norm where its numbers are hard on fp32: repeated calls over
workspaces that hold anything, very large values, means far from zero and
long sums, at sizes of the one-pass kernels and of the streaming ones."""
import math

import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
from oracle import block
from gpu_common import dev, host, say

pytestmark = pytest.mark.gpu
E, EPS = 2.0 ** -24, 1e-5


def _forward(shape, x, gamma, beta, act, ws_fill=0, mx=None, drop=None):
    """(y or (codes, scales), mean, rstd), outputs poisoned before the call."""
    h, w, n, c, g = shape
    gn = mq.mq_norm(h, w, n, c, g, act, EPS)
    mean, rstd = (torch.full((n, g), float("nan"), device="cuda") for _ in range(2))
    ws = torch.full((mq.mqconv_group_norm_workspace_bytes(gn, mq.NORM_FWD),), ws_fill, dtype=torch.uint8, device="cuda")
    if mx is None:
        y = torch.full((h, w, n, c), float("nan"), device="cuda")
        mq.mqconv_group_norm(gn, x, gamma, beta, y, mean, rstd, ws, drop=drop)
        return y, mean, rstd
    t = mq.MxTensor.empty(mq.ROLE_ACT, mx[0], mx[1], (h, w, n, c))
    t.codes.fill_(ws_fill)
    t.scales.fill_(ws_fill)
    mq.mqconv_group_norm_mx(gn, x, gamma, beta, t, mean, rstd, ws, drop=drop)
    return t.codes, t.scales, mean, rstd


def _backward(shape, dy, x, gamma, beta, mean, rstd, act, ws_fill=0, mx=None, drop=None):
    h, w, n, c, g = shape
    gn = mq.mq_norm(h, w, n, c, g, act, EPS)
    dg, db = (torch.full((c,), float("nan"), device="cuda") for _ in range(2))
    ws = torch.full((mq.mqconv_group_norm_workspace_bytes(gn, mq.NORM_BWD),), ws_fill, dtype=torch.uint8, device="cuda")
    if mx is None:
        dx = torch.full((h, w, n, c), float("nan"), device="cuda")
        mq.mqconv_group_norm_backward(gn, dy, x, gamma, beta, mean, rstd, dx, dg, db, ws, drop=drop)
        return dx, dg, db
    t = mq.MxTensor.empty(mq.ROLE_GRAD, mx[0], mx[1], (h, w, n, c))
    t.codes.fill_(ws_fill)
    t.scales.fill_(ws_fill)
    mq.mqconv_group_norm_backward_mx(gn, dy, x, gamma, beta, mean, rstd, t, dg, db, ws, drop=drop)
    return t.codes, t.scales, dg, db


def _random(shape, seed):
    h, w, n, c, _ = shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return r(h, w, n, c), r(h, w, n, c), 1 + 0.2 * r(c), 0.3 * r(c)


@pytest.mark.parametrize("shape", [(16, 16, 2, 32, 8), (19, 23, 5, 90, 9), (20, 20, 128, 256, 32), (80, 80, 16, 64, 16),
                                   (57, 61, 17, 33, 11), (33, 31, 2, 2048, 1), (1, 1, 2000, 24, 3)], ids=str)
def test_calls_repeat_bit_for_bit_whatever_the_workspace_holds(shape):
    say(f"norm repeats {shape}")
    x, dy, gamma, beta = _random(shape, 17)
    drop = mq.mq_drop(0.2, 5)
    ref = None
    for fill in (0x00, 0xFF, 0x7F, 0x01, 0x80):  # zeros, NaN, large values, small ones of both signs
        y = _forward(shape, x, gamma, beta, mq.ACT_SILU, fill, drop=drop)
        got = [*y, *_forward(shape, x, gamma, beta, mq.ACT_SILU, fill, (0, 32), drop),
               *_backward(shape, dy, x, gamma, beta, y[1], y[2], mq.ACT_SILU, fill, drop=drop),
               *_backward(shape, dy, x, gamma, beta, y[1], y[2], mq.ACT_SILU, fill, (1, 32), drop)]
        assert all(bool(torch.isfinite(t).all()) for t in got if t.dtype == torch.float32)
        ref = ref or got
        for i, (a, b) in enumerate(zip(got, ref)):
            assert torch.equal(a, b), f"output {i} differs over a workspace of {fill:#x}"


# one pass; streaming with whole octets, with partial ones, with a group of many workgroups
RANGE_SHAPES = [(16, 16, 4, 32, 8), (13, 7, 3, 24, 3), (64, 64, 4, 64, 16), (57, 61, 17, 33, 11), (33, 31, 2, 2048, 1)]


def _constant_groups(shape, values):
    """Every sample and group holds one value, and what they hold differs."""
    h, w, n, c, g = shape
    v = np.resize(np.asarray(values, np.float32), (n, g))
    return np.broadcast_to(np.repeat(v, c // g, axis=1), (h, w, n, c)).copy(), v


def _equal_to_beta(y, beta):
    np.testing.assert_array_equal(host(y), np.broadcast_to(host(beta), tuple(y.shape)))


@pytest.mark.parametrize("shape", RANGE_SHAPES, ids=str)
def test_large_constant_groups_have_their_value_as_mean(shape):
    """x - mean is 0, so y = beta, however large the value is (its square passes fp32's range from 1.85e19 on)."""
    say(f"norm large constants {shape}")
    _, _, gamma, beta = _random(shape, 3)
    x, v = _constant_groups(shape, [2e19, -1e20, 1.8e19, 3e30])
    y, mean, _ = _forward(shape, dev(x), gamma, beta, mq.ACT_NONE)
    np.testing.assert_array_equal(host(mean), v)
    _equal_to_beta(y, beta)
    _, _, mean, rstd = _forward(shape, dev(x), gamma, beta, mq.ACT_NONE, mx=(0, 32))
    np.testing.assert_array_equal(host(mean), v)
    assert np.isfinite(host(rstd)).all()


@pytest.mark.parametrize("shape", RANGE_SHAPES, ids=str)
def test_deviations_beyond_the_squares_range_give_rstd_0(shape):
    """Deviations from 1e20 to 2e20: their squares are infinite in fp32, rstd is 0 and y = beta; the gradient is 0."""
    say(f"norm large deviations {shape}")
    h, w, n, c, g = shape
    _, dy, gamma, beta = _random(shape, 4)
    rng = np.random.default_rng(4)
    x = (rng.uniform(1e20, 2e20, (h, w, n, c)) * rng.choice([-1, 1], (h, w, n, c))).astype(np.float32)
    ref = x.astype(np.float64).reshape(h * w, n, g, c // g).mean(axis=(0, 3))
    y, mean, rstd = _forward(shape, dev(x), gamma, beta, mq.ACT_NONE)
    # a mean of fp64 sums, rounded once
    assert (np.abs(host(mean) - ref) <= E * np.abs(ref) + 2.0 ** -40 * 2e20).all()
    assert (host(rstd) == 0).all()
    _equal_to_beta(y, beta)
    dx, dgamma, dbeta = _backward(shape, dy, dev(x), gamma, beta, mean, rstd, mq.ACT_NONE)
    assert not host(dx).any() and not host(dgamma).any() and np.isfinite(host(dbeta)).all()


@pytest.mark.parametrize("shape", [*RANGE_SHAPES, (6, 5, 3, 24, 3)], ids=str)
def test_sums_beyond_fp32_of_values_within_it(shape):
    """Groups of 3e38, whose sums of two values already pass fp32's range, and of 1e37, for sums of 64."""
    say(f"norm largest constants {shape}")
    _, _, gamma, beta = _random(shape, 5)
    x, v = _constant_groups(shape, [3e38, 1e37, -3e38, 6e36])
    y, mean, rstd = _forward(shape, dev(x), gamma, beta, mq.ACT_NONE)
    np.testing.assert_array_equal(host(mean), v)
    assert np.isfinite(host(rstd)).all()
    _equal_to_beta(y, beta)


@pytest.mark.parametrize("shape", [*RANGE_SHAPES, (6, 5, 3, 24, 3)], ids=str)
def test_constant_groups_have_variance_0(shape):
    """rstd is 1 / sqrt(eps), one rounding and one of a square root from it, whatever the value."""
    say(f"norm rstd of constants {shape}")
    _, _, gamma, beta = _random(shape, 6)
    x, _ = _constant_groups(shape, [1e6, -3e37, 0.1, 1e20, 7e4])
    _, _, rstd = _forward(shape, dev(x), gamma, beta, mq.ACT_NONE)
    assert (np.abs(host(rstd) * np.sqrt(np.float64(np.float32(EPS))) - 1) <= 2 * E).all()


@pytest.mark.parametrize("ratio", [1e4, 1e6, 5e6])
@pytest.mark.parametrize("shape", RANGE_SHAPES, ids=str)
def test_rstd_keeps_its_digits_at_any_mean(shape, ratio):
    """Squared deviations are fp32 around a mean of at most b values (64 in one pass, 16 streaming): three roundings of each
    and b additions; two roundings as partial results are kept, the rest in fp64. So the variance is within (b + 4) 2^-24, and
    rstd within half of that and a rounding. The values are taken as they are in fp32, with the mean's rounding."""
    say(f"norm far means {shape} {ratio}")
    h, w, n, c, g = shape
    _, _, gamma, beta = _random(shape, 7)
    rng = np.random.default_rng(7)
    far = np.repeat(ratio * rng.uniform(1, 3, (n, g)) * rng.choice([-1, 1], (n, g)), c // g, axis=1)
    x = (rng.standard_normal((h, w, n, c)) + far).astype(np.float32)
    mean, rstd = block.stats(x, g, np.float64(np.float32(EPS)))
    got = _forward(shape, dev(x), gamma, beta, mq.ACT_NONE)
    assert (np.abs(host(got[1]) - mean) <= E * np.abs(mean)).all()
    b = 64 if shape in RANGE_SHAPES[:2] else 16
    err = np.abs(host(got[2]) / rstd - 1)
    assert (err <= ((b + 4) / 2 + 1) * E).all(), f"{err.max():.2e}"


@pytest.mark.parametrize("scale", [1e18, 1e-17])
@pytest.mark.parametrize("shape", [*RANGE_SHAPES, (160, 160, 1, 32, 2)], ids=str)
def test_rstd_of_large_and_small_deviations_whatever_their_number(shape, scale):
    """Squares of 1e36 and 1e-34, whose sums over a group pass fp32's range where they are large: rstd within the bound above
    (eps is 0 for the small ones)."""
    say(f"norm scaled deviations {shape} {scale}")
    h, w, n, c, g = shape
    rng = np.random.default_rng(8)
    x = (scale * rng.uniform(0.5, 1, (h, w, n, c)) * rng.choice([-1, 1], (h, w, n, c))).astype(np.float32)
    eps = 0.0 if scale < 1 else EPS
    gn = mq.mq_norm(h, w, n, c, g, mq.ACT_NONE, eps)
    y, m, r = torch.empty((h, w, n, c), device="cuda"), torch.empty((n, g), device="cuda"), torch.empty((n, g), device="cuda")
    ws = torch.empty(mq.mqconv_group_norm_workspace_bytes(gn, mq.NORM_FWD), dtype=torch.uint8, device="cuda")
    mq.mqconv_group_norm(gn, dev(x), None, None, y, m, r, ws)
    mean, rstd = block.stats(x, g, eps)
    err = np.abs(host(r) / rstd - 1)
    assert (err <= ((64 + 4) / 2 + 1) * E).all(), f"{err.max():.2e}"
    ref = (x - np.repeat(mean, c // g, axis=1)) * np.repeat(rstd, c // g, axis=1)
    # rstd as above, x - mean from a mean rounded to fp32, one rounding of each operation
    assert (np.abs(host(y) - ref) <= 64 * E * np.abs(ref) + 4 * E).all()


@pytest.mark.parametrize("shape", [(160, 160, 8, 256, 32), (64, 64, 128, 512, 64)], ids=str)
def test_long_sums_of_the_gradient(shape):
    """Equal terms in every pixel and sample, whose roundings do not cancel: 100 and 256 of them in a thread. dbeta's terms are
    exact, and a thread's, a chunk's and the whole sum are rounded once each; dgamma's have the rounding of x - mean too."""
    say(f"norm gradient's long sums {shape}")
    h, w, n, c, g = shape
    rng = np.random.default_rng(9)
    xc, gc = rng.standard_normal(c).astype(np.float32), rng.uniform(0.1, 1, c).astype(np.float32)
    x, dy = (dev(v).expand(h, w, n, c).contiguous() for v in (xc, gc))
    _, mean, rstd = _forward(shape, x, None, None, mq.ACT_NONE)
    dx, dgamma, dbeta = _backward(shape, dy, x, None, None, mean, rstd, mq.ACT_NONE)
    m, r = (np.repeat(host(v)[0].astype(np.float64), c // g) for v in (mean, rstd))
    ref_b = gc.astype(np.float64) * (h * w * n)
    ref_g = ref_b * (xc - m) * r
    eb, eg = (np.abs(host(a) / b - 1).max() for a, b in ((dbeta, ref_b), (dgamma, ref_g)))
    say(f"  dbeta {eb / E:.2f}, dgamma {eg / E:.2f} units of 2^-24")
    assert eb <= 3 * E and eg <= 5 * E
    # dx = r (g - mean g - xh mean(g xh)) with the group's means: six roundings of terms of these sizes
    xh = (xc - m) * r
    fold = lambda v: np.repeat(v.reshape(g, -1).mean(axis=1), c // g)  # noqa: E731
    a, b = fold(gc), fold(gc * xh)
    ref = r * (gc - a - xh * b)
    got = host(dx.view(h * w, n, c)[[0, h * w // 2, h * w - 1]])
    assert (np.abs(got - ref) <= 16 * E * r * (gc + a + np.abs(xh) * fold(gc * np.abs(xh)))).all()


@pytest.mark.parametrize("hwn", [(1, 1, 1), (64, 64, 2)], ids=str)
def test_gelu_keeps_its_digits_in_the_tail(hwn):
    """With gamma 0 u is beta exactly: y = u cdf(u), and with dy = 1 dbeta = h w n (cdf(u) + u phi(u)). The argument's rounding
    and its constant's are 1.3 2^-24 of it, (u^2 + 1) times that of cdf; erfc's own error is a few units; phi's argument has three
    roundings of u^2 / 2. Below -12.5 the results are subnormal."""
    h, w, n = hwn
    c = 2048
    u = np.linspace(-12.5, 8, c).astype(np.float32)
    say(f"gelu tail {hwn}")
    shape = (h, w, n, c, 16)
    x, _, _, _ = _random(shape, 10)
    gamma, beta = torch.zeros(c, device="cuda"), dev(u)
    y, mean, rstd = _forward(shape, x, gamma, beta, mq.ACT_GELU)
    v = u.astype(np.float64)
    cdf = np.array([0.5 * math.erfc(-t * math.sqrt(0.5)) for t in v])
    phi = np.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    bound = (1.5 * (v * v + 1) + 16) * E
    got = host(y).reshape(-1, c)
    assert (got == got[0]).all()
    err = np.abs(got[0] - v * cdf) / np.maximum(np.abs(v * cdf), 1e-300)
    assert (err <= bound).all(), f"u = {v[np.argmax(err / bound)]}: {err[np.argmax(err / bound)]:.2e}"
    # 32 values of the tail as a block of their own: its scale is that of the true values
    q = _forward(shape, x, gamma, beta, mq.ACT_GELU, mx=(1, 1))
    scales = host(q[1]).reshape(-1, c // 32)
    top = np.abs((v * cdf).reshape(-1, 32)).max(axis=1)
    clear = np.abs(np.log2(top) - np.round(np.log2(top))) > 1e-3
    assert (scales[:, clear] == (np.floor(np.log2(top)) + 127 - 15).clip(0)[clear]).all()
    dbeta = host(_backward(shape, torch.ones_like(x), x, gamma, beta, mean, rstd, mq.ACT_GELU)[2]) / (h * w * n)
    tol = bound * cdf + (2 * v * v + 16) * E * np.abs(v) * phi
    bad = np.abs(dbeta - (cdf + v * phi)) > tol
    assert not bad.any(), f"u = {v[bad][0]}: {dbeta[bad][0]} for {(cdf + v * phi)[bad][0]}"


def test_silu_keeps_its_digits_in_the_tail():
    """u = beta as above: y = u s(u), dbeta = s (1 + u (1 - s)). exp's argument has a relative rounding of 2^-24 and its
    constant's, the rest a few units; from -88 on the results are tiny or 0."""
    c = 2048
    u = np.linspace(-86, 20, c).astype(np.float32)
    u[:4] = -89, -104, -1e5, -3e38
    say("silu tail")
    shape = (1, 1, 1, c, 16)
    x, _, _, _ = _random(shape, 11)
    gamma, beta = torch.zeros(c, device="cuda"), dev(u)
    y, mean, rstd = _forward(shape, x, gamma, beta, mq.ACT_SILU)
    dbeta = host(_backward(shape, torch.ones_like(x), x, gamma, beta, mean, rstd, mq.ACT_SILU)[2])
    y = host(y).reshape(-1)
    assert (np.abs(y[:4]) <= 1e-36).all() and (np.abs(dbeta[:4]) <= 1e-36).all()
    v, y, dbeta = u[4:].astype(np.float64), y[4:], dbeta[4:]
    s = 1 / (1 + np.exp(-v))
    bound = (1.5 * np.abs(v) + 8) * E
    assert (np.abs(y - v * s) <= bound * np.abs(v * s)).all()
    # 1 - s and 1 + u (1 - s) have roundings of 1 and of u
    assert (np.abs(dbeta - (s + v * s * (1 - s))) <= bound * (s + np.abs(v) * s * (1 - s)) + 4 * E * np.abs(v) * s).all()


def test_gradient_of_more_than_2_to_the_27_channels():
    """One pixel of one sample: dbeta is dy, dgamma dy xh with a rounding of x - mean, of a partial sum and of the result. Eight
    channels a workgroup would be more threads than a launch takes."""
    c, d = 2**27 + 96, 32
    shape = (1, 1, 1, c, c // d)
    say(f"norm gradient of {c} channels")
    x, dy, gamma, beta = _random((1, 1, 1, c, 1), 12)
    _, mean, rstd = _forward(shape, x, gamma, beta, mq.ACT_NONE)
    dx, dgamma, dbeta = _backward(shape, dy, x, gamma, beta, mean, rstd, mq.ACT_NONE)
    codes, scales, dgamma2, dbeta2 = _backward(shape, dy, x, gamma, beta, mean, rstd, mq.ACT_NONE, mx=(1, 32))
    assert torch.equal(dgamma, dgamma2) and torch.equal(dbeta, dbeta2) and torch.equal(dbeta, dy.view(-1))
    ref = mq.MxTensor.empty(mq.ROLE_GRAD, 1, 32, shape[:4])
    mq.mqconv_quantize(dx, ref)
    assert torch.equal(codes, ref.codes) and torch.equal(scales, ref.scales)
    for part in (slice(0, 2**20), slice(c - 2**20, c)):
        m, r = (v.view(-1).repeat_interleave(d)[part].double() for v in (mean, rstd))
        want = dy.view(-1)[part].double() * (x.view(-1)[part].double() - m) * r
        assert bool(((dgamma[part] - want).abs() <= 4 * E * want.abs()).all())
    seg = slice(c - 2**20, c)
    xg, gg = x.view(-1)[seg].double().view(-1, d), (dy.view(-1) * gamma)[seg].double().view(-1, d)
    m, r = mean.view(-1, 1)[-(2**20) // d:].double(), rstd.view(-1, 1)[-(2**20) // d:].double()
    xh = (xg - m) * r
    want = r * (gg - gg.mean(1, keepdim=True) - xh * (gg * xh).mean(1, keepdim=True))
    size = r * (gg.abs() + gg.abs().mean(1, keepdim=True) + xh.abs() * (gg * xh).abs().mean(1, keepdim=True))
    assert bool(((dx.view(-1)[seg].view(-1, d) - want).abs() <= 16 * E * size).all())

"""Layer norm and its gradient on the GPU: fp32 results element by element
against the fp64 oracle, MX results bit for bit against the quantization of the
fp32 ones, non-finite values, in-place calls, odd addresses, streams, graphs and
injected failures.

Bounds, with e = 2^-24, half an fp32 step relative to a value, and sums in fp64
(whose own roundings, 2^-53 a term, disappear in the factor 1.01):
  mean:  e |mean| (+ 1e-13 of the mean |x|: cancelling sums)
  rstd:  e rstd (+ 1e-12)
  y = fma((x - mean) rstd, gamma, beta): the mean's rounding, the subtraction,
  rstd's rounding, the product, the fma:
    |gamma| rstd e (|mean| + 3 |x - mean|) + e |y|
  xh: 2 e |xh| (from the mean and rstd that were kept);  g = gamma dy: e |g|
  k1: e mean|g| + e |k1|;  k2: 3 e mean|g xh| + e |k2|
  t = fma(-xh, k2, g - k1):
    e|g| + dk1 + e |g - k1| + |xh| dk2 + 2 e |xh k2| + e |t|
  dx = rstd t (+ dskip): rstd dt + e |dx|
  dgamma: 2 e of every term, e of the workgroups' fp32 sums, e of the result:
    3 e sum |dy xh| + e |dgamma|;  dbeta: e sum |dy| + e |dbeta|"""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
from oracle import train
from gpu_common import dev, host, say, workspace

pytestmark = pytest.mark.gpu
E, EPS, TINY = 2.0 ** -24, 1e-5, 1e-37

# (H, W, N, C): rows held by 1 to 64 lanes, by a wave in several quads, by 2 to 16 waves, and read in turn; single rows,
# fewer rows than a workgroup holds, many; channels that are no multiple of four
SHAPES = [
    (1, 1, 1, 1), (1, 1, 700, 1), (1, 3, 5, 3), (2, 2, 3, 4), (5, 1, 3, 7), (1, 1, 9, 8), (4, 4, 4, 15), (7, 9, 3, 45),
    (1, 1, 1, 64), (11, 13, 5, 64), (19, 23, 5, 90), (9, 1, 33, 128), (1, 5, 13, 129), (6, 7, 8, 256), (1, 1, 3, 257),
    (3, 3, 7, 512), (2, 1, 5, 700), (1, 2, 9, 1024), (1, 3, 3, 1025), (1, 1, 6, 2048), (2, 2, 3, 3001), (1, 4, 2, 4096),
    (1, 1, 5, 4097), (1, 1, 4, 8192), (1, 1, 3, 8193), (1, 1, 2, 16384), (1, 1, 3, 16385), (1, 2, 1, 50001),
    (40, 41, 6, 32), (64, 64, 16, 20),
]


def _inputs(shape, seed):
    rng = np.random.default_rng(seed)
    c = shape[-1]
    x = (rng.standard_normal(shape) * (0.5 + rng.random(c)) + 0.5 * rng.standard_normal(c)).astype(np.float32)
    dy, skip = (rng.standard_normal(shape).astype(np.float32) for _ in range(2))
    return x, dy, skip, (1 + 0.2 * rng.standard_normal(c)).astype(np.float32), (0.3 * rng.standard_normal(c)).astype(np.float32)


def _nan(*shape):
    return torch.full(shape, float("nan"), device="cuda")


def _mx(role, mx, shape):
    t = mq.MxTensor.empty(role, mx[0], mx[1], shape)
    t.codes.fill_(0xAB)
    t.scales.fill_(0xAB)
    return t


def _forward(shape, x, gamma, beta, mx=None, y=None, residual=None, sum=None, eps=EPS, keep=True, fill=0xFF, stream=None):
    ln = mq.mq_layer_norm(*shape, eps)
    mean, rstd = (_nan(*shape[:3]), _nan(*shape[:3])) if keep else (None, None)
    if mx is None:
        y = _nan(*shape) if y is None else y
        mq.mqconv_layer_norm(ln, x, gamma, beta, y, mean, rstd, residual=residual, sum=sum, stream=stream)
        return y, mean, rstd
    t = _mx(mq.ROLE_ACT, mx, shape)
    ws = workspace(mq.mqconv_layer_norm_workspace_bytes(ln, mq.NORM_FWD)).fill_(fill)
    mq.mqconv_layer_norm_mx(ln, x, gamma, beta, t, mean, rstd, ws, residual=residual, sum=sum, stream=stream)
    return t, mean, rstd


def _backward(shape, dy, x, gamma, mean, rstd, mx=None, dx=None, dskip=None, sums=True, fill=0xFF, stream=None):
    ln = mq.mq_layer_norm(*shape, EPS)
    dg, db = (_nan(shape[3]), _nan(shape[3])) if sums else (None, None)
    ws = workspace(mq.mqconv_layer_norm_workspace_bytes(ln, mq.NORM_BWD)).fill_(fill)
    if mx is None:
        dx = _nan(*shape) if dx is None else dx
        mq.mqconv_layer_norm_backward(ln, dy, x, gamma, mean, rstd, dx, dg, db, ws, dskip=dskip, stream=stream)
        return dx, dg, db
    t = _mx(mq.ROLE_GRAD, mx, shape)
    mq.mqconv_layer_norm_backward_mx(ln, dy, x, gamma, mean, rstd, t, dg, db, ws, dskip=dskip, stream=stream)
    return t, dg, db


def _close(name, got, ref, tol):
    got = np.asarray(got, np.float64)
    assert np.isfinite(got).all(), f"{name}: non-finite"
    bad = np.abs(got - ref) > 1.01 * tol + TINY
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size} beyond the bound, first at {tuple(np.argwhere(bad)[0])}: "
                           f"{got[bad][0]!r} for {ref[bad][0]!r}, bound {np.broadcast_to(tol, ref.shape)[bad][0]:.3e}")


def _check_forward(s, gamma, beta, got, eps=EPS):
    c = s.shape[-1]
    ga = np.ones(c) if gamma is None else gamma.astype(np.float64)
    be = np.zeros(c) if beta is None else beta.astype(np.float64)
    y, mean, rstd = train.layer_norm(s, ga, be, eps)
    s = s.astype(np.float64)
    _close("mean", host(got[1]), mean, E * np.abs(mean) + 1e-13 * np.abs(s).mean(axis=-1))
    _close("rstd", host(got[2]), rstd, (E + 1e-12) * rstd)
    m, r = mean[..., None], rstd[..., None]
    # (where the sum cancels, the mean's error is that of its terms)
    dm = E * np.abs(m) + 1e-13 * np.abs(s).mean(axis=-1, keepdims=True)
    _close("y", host(got[0]), y, np.abs(ga) * r * (dm + 3 * E * np.abs(s - m)) + E * np.abs(y))


def _check_backward(dy, x, gamma, mean, rstd, skip, got):
    ga = np.ones(x.shape[-1]) if gamma is None else gamma.astype(np.float64)
    dx, dgamma, dbeta, q = train.layer_norm_backward(dy, x, ga, mean, rstd, 0.0 if skip is None else skip.astype(np.float64))
    g, xh, k1, k2, r = np.abs(q["g"]), np.abs(q["xh"]), q["k1"], q["k2"], q["r"]
    dk1 = E * g.mean(axis=-1, keepdims=True) + E * np.abs(k1)
    dk2 = 3 * E * (g * xh).mean(axis=-1, keepdims=True) + E * np.abs(k2)
    t = q["g"] - k1 - q["xh"] * k2
    dt = E * g + dk1 + E * np.abs(q["g"] - k1) + xh * dk2 + 2 * E * xh * np.abs(k2) + E * np.abs(t)
    # rstd t is rounded where no skip gradient is added to it exactly
    _close("dx", host(got[0]), dx, r * dt + E * np.abs(dx))
    rows = tuple(range(dy.ndim - 1))
    a = np.abs(dy.astype(np.float64))
    _close("dgamma", host(got[1]), dgamma, 3 * E * (a * xh).sum(axis=rows) + E * np.abs(dgamma))
    _close("dbeta", host(got[2]), dbeta, E * a.sum(axis=rows) + E * np.abs(dbeta))


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward_fp32(shape):
    for affine, extra in ((True, False), (True, True), (False, False)):
        say(f"layer norm {shape} affine={affine} skip={extra}")
        x, dy, skip, gamma, beta = _inputs(shape, sum(shape) + affine)
        if not affine:
            gamma = beta = None
        G, B = (None, None) if gamma is None else (dev(gamma), dev(beta))
        X, DY = dev(x), dev(dy)
        total = None
        if extra:
            total = _nan(*shape)
            got = _forward(shape, X, G, B, residual=dev(skip), sum=total)
            s = x + skip  # fp32: one rounding, the same
            np.testing.assert_array_equal(host(total), s)
        else:
            got = _forward(shape, X, G, B)
            s = x
        _check_forward(s, gamma, beta, got)
        out = _backward(shape, DY, X if total is None else total, G, got[1], got[2], dskip=dev(skip) if extra else None)
        _check_backward(dy, s, gamma, host(got[1]), host(got[2]), skip if extra else None, out)


@pytest.mark.parametrize("shape", [(7, 9, 3, 45), (1, 2, 9, 1024), (1, 1, 3, 16385)], ids=str)
def test_gradient_against_differences(shape):
    """dL/ds of L = sum(dy y) + sum(skip x) along a direction, by fp64 differences of the formula; 1e-4 of the terms' sizes is
    far above fp32's error along it and far below a wrong term."""
    x, dy, skip, gamma, beta = _inputs(shape, 5)
    _, mean, rstd = _forward(shape, dev(x), dev(gamma), dev(beta))
    dx, dg, db = (host(t).astype(np.float64) for t in _backward(shape, dev(dy), dev(x), dev(gamma), mean, rstd, dskip=dev(skip)))
    rng = np.random.default_rng(6)
    v, vg, vb = rng.standard_normal(shape), rng.standard_normal(shape[3]), rng.standard_normal(shape[3])
    f = lambda s: (train.layer_norm(x + s * v, gamma + s * vg, beta + s * vb, EPS)[0] * dy).sum() + (skip * (x + s * v)).sum()  # noqa: E731
    terms = (dx * v, dg * vg, db * vb)
    assert abs((f(1e-4) - f(-1e-4)) / 2e-4 - sum(t.sum() for t in terms)) <= 1e-4 * sum(np.abs(t).sum() for t in terms)


def _columns_close(shape, dy, x, mean, rstd, dgamma, dbeta):
    """dgamma and dbeta against 64-bit sums: 3 e sum |dy xh| + e |dgamma| and e sum |dy| + e |dbeta|, with 2 e of every term's xh."""
    dy, x = host(dy).astype(np.float64).reshape(-1, shape[3]), host(x).astype(np.float64).reshape(-1, shape[3])
    xh = (x - host(mean).astype(np.float64).reshape(-1, 1)) * host(rstd).astype(np.float64).reshape(-1, 1)
    for got, terms, k in ((dgamma, dy * xh, 3), (dbeta, dy, 1)):
        total = terms.sum(axis=0)
        assert (np.abs(host(got) - total) <= k * E * np.abs(terms).sum(axis=0) + E * np.abs(total) + TINY).all()


MX_SHAPES = [(6, 7, 3, 36), (3, 5, 20, 128), (4, 3, 70, 132), (9, 2, 64, 256), (50, 41, 1, 100), (1, 1, 1, 1), (1, 1, 300, 64), (5, 3, 33, 45), (19, 23, 5, 90), (20, 20, 32, 64), (7, 6, 40, 320), (3, 2, 2, 31),
             (2, 3, 37, 1000), (40, 24, 16, 64), (2, 1, 35, 2048), (1, 2, 33, 4100), (1, 3, 3, 9008), (1, 1, 2, 20000)]


def _same_codes(t, ref, label):
    np.testing.assert_array_equal(host(t.scales), host(ref.scales), err_msg=f"scales {label}")
    np.testing.assert_array_equal(host(t.codes), host(ref.codes), err_msg=f"codes {label}")


@pytest.mark.parametrize("shape", MX_SHAPES, ids=str)
@pytest.mark.parametrize("fmt", range(5))
def test_mx_results_are_the_quantized_fp32_results(shape, fmt):
    x, dy, skip, gamma, beta = (dev(a) for a in _inputs(shape, 40 + fmt))
    for bp, extra in ((32, False), (1, True), (32, True), (1, False)):
        say(f"layer norm mx {shape} fmt={fmt} bp={bp} skip={extra}")
        total, total2 = (_nan(*shape), _nan(*shape)) if extra else (None, None)
        y, mean, rstd = _forward(shape, x, gamma, beta, residual=skip if extra else None, sum=total)
        t, mean2, rstd2 = _forward(shape, x, gamma, beta, mx=(fmt, bp), residual=skip if extra else None, sum=total2)
        assert torch.equal(mean, mean2) and torch.equal(rstd, rstd2) and (not extra or torch.equal(total, total2))
        ref = mq.MxTensor.empty(mq.ROLE_ACT, fmt, bp, shape)
        mq.mqconv_quantize(y, ref)
        _same_codes(t, ref, f"y {shape}")
        t, _, _ = _forward(shape, x, gamma, beta, mx=(fmt, bp), residual=skip if extra else None, sum=total2, keep=False, fill=0)
        _same_codes(t, ref, f"y without statistics {shape}")
        s = total if extra else x
        dx, dg, db = _backward(shape, dy, s, gamma, mean, rstd, dskip=skip if extra else None)
        t, dg2, db2 = _backward(shape, dy, s, gamma, mean, rstd, mx=(fmt, bp), dskip=skip if extra else None, fill=0)
        # (the two forms share the rows between workgroups in their own ways: both within the bound of 64-bit sums)
        _columns_close(shape, dy, s, mean, rstd, dg2, db2)
        ref = mq.MxTensor.empty(mq.ROLE_GRAD, fmt, bp, shape)
        mq.mqconv_quantize(dx, ref)
        _same_codes(t, ref, f"dx {shape}")


SOME = [(7, 9, 3, 45), (16, 16, 4, 64), (1, 3, 5, 1024), (1, 2, 3, 5000), (1, 1, 3, 20000)]


@pytest.mark.parametrize("shape", SOME, ids=str)
def test_a_mean_far_from_zero_keeps_its_digits(shape):
    """x = 3000 + noise: sums of squares around zero in fp32 would lose the variance."""
    x, _, _, gamma, beta = _inputs(shape, 8)
    x = (x + np.float32(3000)).astype(np.float32)
    _check_forward(x, gamma, beta, _forward(shape, dev(x), dev(gamma), dev(beta)))


@pytest.mark.parametrize("shape", SOME, ids=str)
@pytest.mark.parametrize("size", [1e19, 1e30, 1e-19, 1e-30])
def test_large_and_small_values(shape, size):
    """Squares of these leave fp32's range on either side: sums are fp64. (eps is scaled with the values.)"""
    x, _, _, gamma, beta = _inputs(shape, 9)
    x = (x * np.float32(size)).astype(np.float32)
    eps = float(np.float32(min(1e-5 * size * size, 1e30)))
    _check_forward(x, gamma, beta, _forward(shape, dev(x), dev(gamma), dev(beta), eps=eps), eps=eps)


@pytest.mark.parametrize("shape", SOME, ids=str)
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_non_finite_values_stay_in_their_row(shape, value):
    x, dy, _, gamma, beta = _inputs(shape, 12)
    G, B = dev(gamma), dev(beta)
    clean = _forward(shape, dev(x), G, B)
    ref = _backward(shape, dev(dy), dev(x), G, clean[1], clean[2])
    x[0, -1, 2, 5] = value
    got = _forward(shape, dev(x), G, B)
    out = _backward(shape, dev(dy), dev(x), G, got[1], got[2])
    inside = np.zeros(shape, bool)
    inside[0, -1, 2] = True
    for name, a, b in (("y", got[0], clean[0]), ("dx", out[0], ref[0])):
        a, b = host(a), host(b)
        assert np.isnan(a[inside]).all(), name
        np.testing.assert_array_equal(a[~inside], b[~inside], err_msg=name)
    assert np.isnan(host(got[2])[0, -1, 2]) and np.isnan(host(out[1])).all() and np.isfinite(host(out[2])).all()
    t, _, _ = _forward(shape, dev(x), G, B, mx=(0, 32))
    q = mq.MxTensor.empty(mq.ROLE_ACT, 0, 32, shape)
    mq.mqconv_quantize(got[0], q)
    _same_codes(t, q, "non-finite")


def test_constant_rows_and_zero_gradients():
    shape = (6, 5, 3, 16)
    x = np.full(shape, 2.5, np.float32)
    _, dy, _, gamma, beta = _inputs(shape, 3)
    y, mean, rstd = _forward(shape, dev(x), dev(gamma), dev(beta))
    assert (host(mean) == 2.5).all()
    np.testing.assert_array_equal(host(y), np.broadcast_to(beta, shape))
    dx, dg, db = _backward(shape, dev(np.zeros_like(x)), dev(x), dev(gamma), mean, rstd)
    assert not host(dx).any() and not host(dg).any() and not host(db).any()
    y, _, rstd = _forward(shape, dev(x), dev(gamma), dev(beta), eps=0.0)
    assert np.isinf(host(rstd)).all() and np.isnan(host(y)).all()


@pytest.mark.parametrize("shape", SOME, ids=str)
def test_in_place_optional_outputs_and_another_stream(shape):
    say(f"layer norm in place {shape}")
    x, dy, skip, gamma, beta = (dev(a) for a in _inputs(shape, 21))
    s0 = _nan(*shape)
    y, mean, rstd = _forward(shape, x, gamma, beta, residual=skip, sum=s0)
    dx, dg, db = _backward(shape, dy, s0, gamma, mean, rstd, dskip=skip)
    for which in range(4):  # sum over x or the residual, y over the other
        a, b = x.clone(), skip.clone()
        total, out = (a, b) if which & 1 else (b, a)
        if which & 2:
            total = _nan(*shape)
        _forward(shape, a, gamma, beta, residual=b, sum=total, y=out)
        assert torch.equal(out, y) and torch.equal(total, s0)
    for which in range(3):
        a, b, c = dy.clone(), s0.clone(), skip.clone()
        out = (a, b, c)[which]
        got = _backward(shape, a, b, gamma, mean, rstd, dskip=c, dx=out)
        assert torch.equal(out, dx) and torch.equal(got[1], dg) and torch.equal(got[2], db)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2, dx2, s2 = torch.empty_like(y), torch.empty_like(dx), _nan(*shape)
    torch.cuda.synchronize()
    _forward(shape, x, gamma, beta, residual=skip, sum=s2, y=y2, keep=False, stream=st)
    ln = mq.mq_layer_norm(*shape, EPS)
    ws = workspace(mq.mqconv_layer_norm_workspace_bytes(ln, mq.NORM_BWD))
    mq.mqconv_layer_norm_backward(ln, dy, s0, gamma, mean, rstd, dx2, ws=ws, dskip=skip, stream=st)
    st.synchronize()
    assert torch.equal(y2, y) and torch.equal(dx2, dx)


@pytest.mark.parametrize("shape", SOME, ids=str)
def test_any_four_byte_address_and_nothing_behind_the_tensors(shape):
    x, dy, skip, gamma, beta = _inputs(shape, 23)
    aligned = _forward(shape, dev(x), dev(gamma), dev(beta))
    ref = _backward(shape, dev(dy), dev(x), dev(gamma), aligned[1], aligned[2], dskip=dev(skip))

    def odd(a):
        big = torch.full((a.size + 9,), 7.0, device="cuda")
        view = big[1:1 + a.size]
        view.copy_(torch.from_numpy(a.reshape(-1)))
        return big, view

    views = [odd(a) for a in (x, dy, skip, gamma, beta)]
    X, DY, SK, G, B = (v for _, v in views)
    outs = [odd(np.zeros(shape, np.float32)) for _ in range(2)]
    stats = [odd(np.zeros(shape[:3], np.float32)) for _ in range(2)]
    sums = [odd(np.zeros(shape[3], np.float32)) for _ in range(2)]
    ln = mq.mq_layer_norm(*shape, EPS)
    mq.mqconv_layer_norm(ln, X, G, B, outs[0][1], stats[0][1], stats[1][1])
    ws = workspace(mq.mqconv_layer_norm_workspace_bytes(ln, mq.NORM_BWD))
    mq.mqconv_layer_norm_backward(ln, DY, X, G, stats[0][1], stats[1][1], outs[1][1], sums[0][1], sums[1][1], ws, dskip=SK)
    pairs = ((outs[0], aligned[0]), (stats[0], aligned[1]), (stats[1], aligned[2]), (outs[1], ref[0]), (sums[0], ref[1]),
             (sums[1], ref[2]))
    for (big, view), r in pairs:
        assert torch.equal(view, r.reshape(-1))
        assert (big[:1] == 7).all() and (big[1 + r.numel():] == 7).all()


@pytest.mark.parametrize("shape", [(16, 16, 4, 64), (1, 2, 9, 1024), (1, 1, 3, 20000)], ids=str)
def test_graph_replays_are_the_eager_results(shape):
    x, dy, skip, gamma, beta = (dev(a) for a in _inputs(shape, 30))
    ln = mq.mq_layer_norm(*shape, EPS)
    y, dx, total = (torch.empty_like(x) for _ in range(3))
    mean, rstd = torch.empty(*shape[:3], device="cuda"), torch.empty(*shape[:3], device="cuda")
    dg, db = torch.empty(shape[3], device="cuda"), torch.empty(shape[3], device="cuda")
    yq, dxq = mq.MxTensor.empty(mq.ROLE_ACT, 4, 32, shape), mq.MxTensor.empty(mq.ROLE_GRAD, 1, 1, shape)
    ws = workspace(max(mq.mqconv_layer_norm_workspace_bytes(ln, k) for k in (0, 1)))
    outs = (y, total, mean, rstd, dx, dg, db, yq.codes, yq.scales, dxq.codes, dxq.scales)

    def path():
        mq.mqconv_layer_norm(ln, x, gamma, beta, y, mean, rstd, residual=skip, sum=total)
        mq.mqconv_layer_norm_mx(ln, x, gamma, beta, yq, ws=ws, residual=skip, sum=total)
        mq.mqconv_layer_norm_backward(ln, dy, total, gamma, mean, rstd, dx, dg, db, ws, dskip=skip)
        mq.mqconv_layer_norm_backward_mx(ln, dy, total, gamma, mean, rstd, dxq, dg, db, ws, dskip=skip)

    eager = []
    for k in range(3):
        x.mul_(1.5)
        path()
        eager.append([x.clone()] + [t.clone() for t in outs])
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        path()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            path()
    for k in (1, 0, 2, 2, 1):
        for t in outs:
            t.fill_(0x5A if t.dtype == torch.uint8 else float("nan"))
        x.copy_(eager[k][0])
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        for i, (t, e) in enumerate(zip(outs, eager[k][1:])):
            assert torch.equal(t, e), f"replay {k}: output {i} differs"
        path()


def test_repeats_bit_for_bit_and_injected_failures():
    shape = (16, 16, 4, 64)
    x, dy, skip, gamma, beta = (dev(a) for a in _inputs(shape, 33))
    calls = (lambda f=0: _forward(shape, x, gamma, beta, mx=(0, 32), fill=f),
             lambda f=0: _backward(shape, dy, x, gamma, *_forward(shape, x, gamma, beta)[1:], mx=(1, 32), fill=f))
    refs = [c() for c in calls]
    for c, ref in zip(calls, refs):
        for fill in (0xFF, 0x7F, 1):
            got = c(fill)
            _same_codes(got[0], ref[0], f"workspace of {fill}")
            assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])
    try:
        for c, ref, launches in zip(calls, refs, (1, 3)):
            for k in range(1, launches + 2):
                mq.mqconv_inject_launch_failure(k)
                if k <= launches:
                    with pytest.raises(mq.MqConvError) as e:
                        c()
                    assert e.value.status == -7
                else:
                    got = c()
                    mq.mqconv_inject_launch_failure(0)
                    _same_codes(got[0], ref[0], "after failures")
                    assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])
    finally:
        mq.mqconv_inject_launch_failure(0)


@pytest.mark.parametrize("shape", [(6, 7, 3, 36), (3, 2, 33, 64), (9, 2, 64, 256), (4, 3, 5, 320)], ids=str)
@pytest.mark.parametrize("bp", [1, 32])
def test_mx_results_of_non_finite_rows(shape, bp):
    """A row with a NaN or an infinity is NaN in the fp32 form; the MX form is what the quantizer makes of that."""
    x, dy, skip, gamma, beta = _inputs(shape, 71)
    x[0, 0, 0, -1], x[-1, -1, -1, 0], x[1, 1, 1, 5] = np.nan, np.inf, -np.inf
    x, dy, gamma, beta = dev(x), dev(dy), dev(gamma), dev(beta)
    y, mean, rstd = _forward(shape, x, gamma, beta)
    for fmt in (0, 1, 2, 4):
        t, _, _ = _forward(shape, x, gamma, beta, mx=(fmt, bp))
        ref = mq.MxTensor.empty(mq.ROLE_ACT, fmt, bp, shape)
        mq.mqconv_quantize(y, ref)
        _same_codes(t, ref, f"y {shape}")
        dx, _, _ = _backward(shape, dy, x, gamma, mean, rstd)
        t, _, _ = _backward(shape, dy, x, gamma, mean, rstd, mx=(fmt, bp), sums=False)
        ref = mq.MxTensor.empty(mq.ROLE_GRAD, fmt, bp, shape)
        mq.mqconv_quantize(dx, ref)
        _same_codes(t, ref, f"dx {shape}")

"""The orthogonalised weight update on the GPU against the fp64 oracle.

One step is held to an elementwise bound. With d = 2^-22, what two f16 parts
lose of a value (each rounds by at most 2^-11 of what it rounds) and what leaving
out the product of two low parts loses, e = 2^-24, and G(k) = (k + 3) e for a
sum of k products in fp32 in any order, and |.| elementwise:
  X0: e + d of it =: d0
  S = X X^T:         dS = (2 d0 + d + G(n)) |X| |X|^T + d |S|
  S^2:               dQ = |S| dS + dS |S| + (d + G(m)) |S| |S|
  F = a I + b S + c S^2:  dF = |b| dS + |c| dQ + 4 e (|a| I + |b| |S| + |c| |S| |S|) + d |F|
  X1 = F X:          (dF + (d0 + d + G(m)) |F|) |X| + e |X1|
Values below 2^-39 are stored with an absolute error: 2^-40 is added to every d.

Several steps are held to a model of their rounding: the same steps in fp64,
every stored matrix rounded to 20 bits (a random rounding of each value by up to
2^-20 of it, 4 times what the kernel's stored values lose, which also covers its
fp32 sums: their errors grow with the square root of the number of 16-product
blocks, 2^-25 sqrt(k / 16) of the terms' root mean square, below 2^-21 for the
k <= 4096 here), may differ from the exact ones by R in the 2-norm; the kernel
may by 2 R, and by 2 max + 6 rms of the model's errors in an element."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
from oracle import train
from gpu_common import dev, host, say, workspace

pytestmark = pytest.mark.gpu
E, D = 2.0 ** -24, 2.0 ** -22
MUON = (3.4445, -4.7750, 2.0315)
f32 = lambda v: float(np.float32(v))  # noqa: E731

# single values, vectors both ways, one tile and its neighbours, extents below and above multiples of 32, 64 and 128, several
# tiles on both sides of the diagonal, tall and wide
SHAPES = [(1, 1), (1, 37), (37, 1), (2, 3), (16, 27), (27, 16), (31, 33), (32, 32), (33, 31), (64, 64), (65, 64), (63, 130),
          (64, 576), (576, 64), (100, 300), (129, 127), (200, 457), (257, 129)]


def _gradient(shape, seed, kind="mixed"):
    rng = np.random.default_rng(seed)
    m, n = shape
    if kind == "noise":
        g = rng.standard_normal(shape)
    elif kind == "rank1":
        g = np.outer(rng.standard_normal(m), rng.standard_normal(n))
    else:  # a few strong directions and noise, as gradients are
        r = max(1, min(m, n) // 8)
        g = rng.standard_normal((m, r)) @ (rng.standard_normal((r, n)) * np.logspace(0, -2, r)[:, None]) + 0.3 * rng.standard_normal(shape)
    return (1e-3 * g).astype(np.float32)


def _run(newton, mats, out=None, fill=0xFF, stream=None):
    u = [dev(g) for g in mats]
    x = [torch.full(tuple(g.shape), float("nan"), device="cuda") for g in mats] if out is None else out(u)
    ws = workspace(mq.mqconv_orthogonalize_workspace_bytes([g.shape for g in mats])).fill_(fill)
    mq.mqconv_orthogonalize(newton, u, x, ws, stream=stream)
    return [host(t) for t in x]


def _one_step_bound(g, a, b, c, eps):
    tall = g.shape[0] > g.shape[1]
    x = np.asarray(g.T if tall else g, np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    m, n = x.shape
    tiny, G = 2.0 ** -40, lambda k: (k + 3) * E  # noqa: E731
    ax = np.abs(x)
    dx = (E + D) * ax + tiny
    s = x @ x.T
    ds = dx @ ax.T + ax @ dx.T + (D + G(n)) * (ax @ ax.T) + D * np.abs(s) + tiny
    as_ = np.abs(s)
    dq = as_ @ ds + ds @ as_ + (D + G(m)) * (as_ @ as_)
    f = a * np.eye(m) + b * s + c * (s @ s)
    df = abs(b) * ds + abs(c) * dq + 4 * E * (abs(a) * np.eye(m) + abs(b) * as_ + abs(c) * (as_ @ as_)) + D * np.abs(f) + tiny
    ref = f @ x
    tol = df @ ax + np.abs(f) @ dx + (D + G(m)) * (np.abs(f) @ ax) + E * np.abs(ref) + tiny
    return (ref.T, tol.T) if tall else (ref, tol)


@pytest.mark.parametrize("coef", [MUON, (1.5, -0.5, 0.0)], ids=["quintic", "cubic"])
def test_one_step_element_by_element(coef):
    coef = tuple(f32(v) for v in coef)
    for k, shape in enumerate(SHAPES):
        for kind in ("mixed", "noise", "rank1"):
            g = _gradient(shape, 100 + k, kind)
            got = _run(mq.mq_newton(1, *coef, 1e-7), [g])[0]
            ref, tol = _one_step_bound(g, *coef, f32(1e-7))
            bad = ~(np.abs(got - ref) <= 1.01 * tol)
            say(f"one step {shape} {kind}: {np.abs(got - ref).max():.2e}, of the bound {np.max(np.abs(got - ref) / tol):.2f}")
            assert not bad.any(), f"{shape} {kind}: {bad.sum()} beyond the bound, first at {tuple(np.argwhere(bad)[0])}"


def _check_model(got, ref, model, label):
    """A single singular value (a vector) gives the model one number, which may be exact by chance, so vectors are held to the
    worst case instead. From x = 1 the quintic steps lead to 0.70, 1.11, 0.72, 1.11, 0.72. A step's factor F = a + b S + c S^2
    is off by 3 d (|b| S + 2 |c| S^2) / F of itself, 3 d for S = x^2 and its rounding: 38 d at x = 1 (F = 0.70), 6 d at 0.7
    (F = 1.59), 56 d at 1.11 (F = 0.65); what x is off grows by |x p'(x) / p(x)| = 0.7 at 0.7 and 2.0 at 1.11. In all
    ((((38 * 0.7 + 6) * 2 + 56) * 0.7 + 6) * 2 + 56) = 238 d, and less than 300 d with the roundings of x itself."""
    err, mod = got - ref, model - ref
    if min(ref.shape) == 1:
        assert (np.abs(err) <= 300 * D * np.abs(ref) + 2.0 ** -40).all(), label
        return
    r = np.linalg.norm(mod)
    say(f"{label}: relative error {np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300):.2e}, model {r / max(np.linalg.norm(ref), 1e-300):.2e}")
    floor = 1e-6 * np.linalg.norm(ref) / np.sqrt(ref.size)  # (a model of few values may be exact by chance)
    assert np.isfinite(got).all() and np.linalg.norm(err) <= 2 * r + floor * np.sqrt(ref.size), label
    assert np.abs(err).max() <= 2 * np.abs(mod).max() + 6 * r / np.sqrt(ref.size) + 8 * floor, label


@pytest.mark.parametrize("kind", ["mixed", "noise"])
def test_five_steps_of_every_shape_in_one_call(kind):
    """All shapes share the launches of one call; each result is that of a call of its own, bit for bit."""
    mats = [_gradient(s, 7 + k, kind) for k, s in enumerate(SHAPES)]
    nt = mq.mq_newton()
    args = (5, nt.a, nt.b, nt.c, nt.eps)
    got = _run(nt, mats)
    for g, x in zip(mats, got):
        _check_model(x.astype(np.float64), train.newton(g, *args), train.newton(g, *args, bits=20), f"five steps {g.shape} {kind}")
        np.testing.assert_array_equal(_run(nt, [g], fill=0)[0], x)


@pytest.mark.parametrize("shape", [(1024, 1024), (1100, 2050), (1536, 640), (1550, 2600), (1800, 1800), (48, 7000), (6400, 300)], ids=str)
def test_large_matrices(shape):
    nt = mq.mq_newton()
    args = (5, nt.a, nt.b, nt.c, nt.eps)
    g = _gradient(shape, 3)
    got = _run(nt, [g])[0]
    _check_model(got.astype(np.float64), train.newton(g, *args), train.newton(g, *args, bits=20), f"large {shape}")
    # converged cubic steps: the rows of the smaller side are orthonormal
    q = _run(mq.mq_newton(32, 1.5, -0.5, 0.0, 0.0), [_gradient(shape, 4, "noise")])[0].astype(np.float64)
    q = q if shape[0] <= shape[1] else q.T
    if shape[0] != shape[1]:  # (a square noise matrix has singular values near 0)
        assert np.abs(q @ q.T - np.eye(len(q))).max() < 1e-4


def test_scales_of_the_input_and_special_values():
    nt = mq.mq_newton(5, eps=0.0)
    args = (5, nt.a, nt.b, nt.c, 0.0)
    g = _gradient((48, 80), 11)
    for size in (1e-30, 1e-10, 1e10, 1e38):  # |U|^2 leaves fp32's range
        h = (g / np.abs(g).max() * size).astype(np.float32)
        _check_model(_run(nt, [h])[0].astype(np.float64), train.newton(h, *args), train.newton(h, *args, bits=20), f"size {size}")
    assert not _run(mq.mq_newton(), [np.zeros((48, 80), np.float32)])[0].any()
    assert np.isnan(_run(nt, [np.zeros((48, 80), np.float32)])[0]).all()
    clean = _run(nt, [g])[0]
    for value in (np.nan, np.inf, -np.inf):  # a bad matrix leaves the others of its call alone
        bad = g.copy()
        bad[3, 70] = value
        a, b, c = _run(nt, [g, bad, g])
        assert np.isnan(b).all()
        np.testing.assert_array_equal(a, clean)
        np.testing.assert_array_equal(c, clean)


def test_in_place_strange_addresses_another_stream_and_repeats():
    mats = [_gradient(s, 31 + k) for k, s in enumerate([(37, 70), (130, 33), (5, 1)])]
    nt = mq.mq_newton()
    ref = _run(nt, mats)
    for a, b in zip(_run(nt, mats, out=lambda u: u, fill=0x7F), ref):
        np.testing.assert_array_equal(a, b)
    bigs = [torch.full((g.size + 9,), 7.0, device="cuda") for g in mats]
    ins = [torch.full((g.size + 9,), 7.0, device="cuda") for g in mats]
    u = [t[1:1 + g.size].view(g.shape) for t, g in zip(ins, mats)]
    x = [t[3:3 + g.size].view(g.shape) for t, g in zip(bigs, mats)]
    for t, g in zip(u, mats):
        t.copy_(dev(g))
    ws = workspace(mq.mqconv_orthogonalize_workspace_bytes([g.shape for g in mats]))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    mq.mqconv_orthogonalize(nt, u, x, ws, stream=st)
    st.synchronize()
    for t, v, r in zip(bigs, x, ref):
        np.testing.assert_array_equal(host(v), r)
        assert (host(t[:3]) == 7).all() and (host(t[3 + r.size:]) == 7).all()


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("scale", [0, 1, 2])
def test_muon_update(nesterov, scale):
    shapes = [(16, 27), (130, 64), (64, 3, 3, 64), (1, 5), (70, 200)]
    rng = np.random.default_rng(scale)
    flat = lambda a: a.reshape(a.shape[0], -1)  # noqa: E731
    g, m = ([_gradient((s[0], int(np.prod(s[1:]))), 50 + 10 * j + k).reshape(s) for k, s in enumerate(shapes)] for j in range(2))
    w = [rng.standard_normal(s).astype(np.float32) * np.float32(0.1) for s in shapes]
    G, M, W = ([dev(a) for a in t] for t in (g, m, w))
    opt = mq.mq_muon(0.02, 0.95, 0.1, nesterov, scale)
    rate = torch.tensor([0.5], device="cuda")
    opt2 = mq.mq_muon(0.04, 0.95, 0.1, nesterov, scale, rate=rate)
    ws = workspace(mq.mqconv_orthogonalize_workspace_bytes(shapes))
    M2, W2 = [t.clone() for t in M], [t.clone() for t in W]
    mq.mqconv_muon_update(opt, G, M, W, ws)
    mq.mqconv_muon_update(opt2, G, M2, W2, ws)
    nt = opt.newton
    args = (5, nt.a, nt.b, nt.c, nt.eps)
    lr, mu, wd = opt.lr, opt.momentum, opt.decay
    for i, s in enumerate(shapes):
        np.testing.assert_array_equal(host(G[i]), g[i])
        assert torch.equal(M[i], M2[i]) and torch.equal(W[i], W2[i])  # 0.04 * 0.5: the same rate
        om, ow = train.muon(flat(g[i]), flat(m[i]), flat(w[i]), lr, mu, wd, nesterov, scale, args)
        _, model = train.muon(flat(g[i]), flat(m[i]), flat(w[i]), lr, mu, wd, nesterov, scale, args, bits=20)
        assert (np.abs(flat(host(M[i])) - om) <= 1.01 * E * np.abs(om) + 1e-40).all()
        err, mod = flat(host(W[i])).astype(np.float64) - ow, model - ow
        step = np.abs(ow - (1 - lr * wd) * flat(w[i]))
        # the roundings of w times its factor, of that factor, of the sum and of the step's factor
        own = E * (3 * np.abs(flat(w[i])) + np.abs(ow) + 4 * step)
        assert (np.abs(err) <= 2 * np.abs(mod).max() + 6 * np.sqrt((mod ** 2).mean()) + 1.01 * own + 1e-6 * step).all()
        say(f"muon {s} nesterov={nesterov} scale={scale}: {np.abs(err).max():.2e}")


def test_captured_updates_follow_the_rate():
    shapes = [(64, 130), (33, 20)]
    g, m, w = ([dev(_gradient(s, 70 + 10 * j + k)) for k, s in enumerate(shapes)] for j in range(3))
    rate = torch.ones(1, device="cuda")
    opt = mq.mq_muon(0.02, 0.9, 0.01, True, mq.MUON_SCALE_RMS, rate=rate)
    ws = workspace(mq.mqconv_orthogonalize_workspace_bytes(shapes))
    start = [[t.clone() for t in v] for v in (m, w)]

    def reset():
        for v, s in zip((m, w), start):
            for t, b in zip(v, s):
                t.copy_(b)

    def path():
        mq.mqconv_muon_update(opt, g, m, w, ws)

    eager = []
    for r in (1.0, 0.25, 3.0):
        rate.fill_(r)
        path()
        eager.append([t.clone() for v in (m, w) for t in v])
    reset()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        path()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            path()
    for again in range(2):
        reset()
        for r, ref in zip((1.0, 0.25, 3.0), eager):
            rate.fill_(r)
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                graph.replay()
            torch.cuda.synchronize()
            for t, e in zip([t for v in (m, w) for t in v], ref):
                assert torch.equal(t, e)
        ws.fill_(0xFF)


def test_injected_failures_then_recovery():
    g = _gradient((70, 40), 90)
    nt = mq.mq_newton(2)
    ref = _run(nt, [g])[0]
    try:
        for k in range(1, 10):
            mq.mqconv_inject_launch_failure(k)
            if k <= 8:  # norm, start, two steps of three products
                with pytest.raises(mq.MqConvError) as e:
                    _run(nt, [g])
                assert e.value.status == -7
            else:
                got = _run(nt, [g])[0]
                mq.mqconv_inject_launch_failure(0)
                np.testing.assert_array_equal(got, ref)
    finally:
        mq.mqconv_inject_launch_failure(0)

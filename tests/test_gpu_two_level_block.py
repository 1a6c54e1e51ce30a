"""The operators of a layer trained in the two-level format one after the
other, as the example uses them: it runs, one step's results are the oracle's
(each stage from what the GPU gave the next one, with the bounds of the single
operators), its gradients are those of differences, and a captured step replays
to the eager results."""
import os
import sys

import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
import oracle
from oracle import train
from gpu_common import dev, host, say
from test_gpu_layer_norm import _check_backward, _check_forward
from test_gpu_nvfp_gemm import _close
from test_gpu_update import _check_model

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import two_level_block  # noqa: E402

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def _inputs(n, size, c):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((size, size, n, c)).astype(np.float32)
    return x, (1e-2 * rng.standard_normal(x.shape)).astype(np.float32)


def _values(role, t):
    return oracle.nvfp_dequantize(role, mq.E2M1, *oracle.nvfp_quantize(role, mq.E2M1, t))


def test_it_runs():
    losses = two_level_block.train(steps=3, n=8, size=6, c=32)
    say("two-level block losses " + " ".join(f"{v:.3f}" for v in losses))
    assert all(np.isfinite(losses))


@pytest.mark.parametrize("n, size, c", [(12, 7, 64), (5, 6, 45), (64, 8, 64)])
def test_one_step_against_the_oracle(n, size, c):
    b = two_level_block.Block(n, size, c, seed=5)
    x, dy = _inputs(n, size, c)
    X, DY = dev(x), dev(dy)
    y = host(b.forward(X)).copy()
    b.backward(X, DY)
    gamma, beta, w = host(b.gamma).copy(), host(b.beta).copy(), host(b.w).copy()
    _check_forward(x, gamma, beta, (b.h, b.mean, b.rstd))
    s = (n, c, size, size, c, 3, 3, 1, 1, 1, 1)
    hv, wv, gv = _values(mq.ROLE_ACT, host(b.h)), _values(mq.ROLE_WEIGHT, w), _values(mq.ROLE_GRAD, dy)
    conv = torch.empty_like(b.y)
    mq.mqconv_nvfp_forward(b.shape, b.hq, b.wq, conv, b.ws)
    _close(s, 0, host(conv), hv, wv, "block")
    np.testing.assert_array_equal(y, host(conv) + x)
    _close(s, 2, host(b.dw), gv, hv, "block")
    _close(s, 1, host(b.dh), gv, wv, "block")
    _check_backward(host(b.dh), x, gamma, host(b.mean), host(b.rstd), dy, (b.dx, b.dgamma, b.dbeta))
    dw, nt = host(b.dw).reshape(c, -1), b.muon.newton
    b.step()
    args = (nt.steps, nt.a, nt.b, nt.c, nt.eps)
    f = lambda v: float(np.float32(v))  # noqa: E731
    old, lr = w.astype(np.float64).reshape(c, -1), f(0.05)
    m, new = train.muon(dw, np.zeros_like(dw), old, lr, f(0.9), 0.0, True, 1, args)
    model = train.muon(dw, np.zeros_like(dw), old, lr, f(0.9), 0.0, True, 1, args, bits=20)[1]
    assert (np.abs(host(b.momentum).reshape(c, -1) - m) <= E * np.abs(m)).all()
    # what the weight moved by, over lr: its own rounding is e |w| / lr, which the bound of the steps does not hold
    moved = (host(b.w).reshape(c, -1).astype(np.float64) - old) / lr
    rounding = E * np.abs(new) / lr
    ref, mod = (new - old) / lr, (model - old) / lr
    clipped = ref + np.sign(moved - ref) * np.maximum(np.abs(moved - ref) - 1.01 * rounding, 0.0)
    _check_model(clipped, ref, mod, f"block {c}")


def test_gradients_are_those_of_differences():
    """d(sum dy (x + conv(LN(x)))) along a direction of x, gamma and beta, with the weight's and the gradient's values as they
    are quantized and the activation in fp64 (its quantization has no derivative). dh, the gradient that reaches the norm, is
    that of the quantized dy; the skip path has dy itself. 1e-4 of the terms' sizes: far above fp32's error along the direction
    and the differences', far below a wrong term."""
    n, size, c = 6, 5, 32
    b = two_level_block.Block(n, size, c, seed=9)
    x, dy = _inputs(n, size, c)
    X, DY = dev(x), dev(dy)
    b.forward(X)
    b.backward(X, DY)
    gamma, beta = host(b.gamma).astype(np.float64), host(b.beta).astype(np.float64)
    wv, gv = _values(mq.ROLE_WEIGHT, host(b.w)), _values(mq.ROLE_GRAD, dy)
    rng = np.random.default_rng(3)
    v, vg, vb = rng.standard_normal(x.shape), rng.standard_normal(c), rng.standard_normal(c)

    def f(t):
        h = train.layer_norm(x + t * v, gamma + t * vg, beta + t * vb, 1e-5)[0]
        return (gv * oracle.conv_fwd(b.shape, h, wv)).sum() + (dy * (x + t * v)).sum()

    terms = (host(b.dx) * v, host(b.dgamma) * vg, host(b.dbeta) * vb)
    assert abs((f(1e-4) - f(-1e-4)) / 2e-4 - sum(t.sum() for t in terms)) <= 1e-4 * sum(np.abs(t).sum() for t in terms)


def test_a_captured_step_replays_to_the_eager_results():
    n, size, c = 16, 8, 64
    x, dy = _inputs(n, size, c)
    X, DY = dev(x), dev(dy)

    def state(b):
        return [t.clone() for t in (b.y, b.dx, b.dw, b.dgamma, b.dbeta, b.w, b.momentum, b.gamma, b.beta)]

    eager, steps = two_level_block.Block(n, size, c, seed=2), []
    for _ in range(4):
        eager.forward(X)
        eager.backward(X, DY)
        eager.step()
        steps.append(state(eager))
    b = two_level_block.Block(n, size, c, seed=2)
    start = [t.clone() for t in (b.w, b.momentum, b.gamma, b.beta)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        b.forward(X)
        b.backward(X, DY)
        b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        b.forward(X)
        b.backward(X, DY)
        b.step()
    for t, s in zip((b.w, b.momentum, b.gamma, b.beta), start):
        t.copy_(s)
    for k, ref in enumerate(steps):
        graph.replay()
        torch.cuda.synchronize()
        for i, (got, want) in enumerate(zip(state(b), ref)):
            assert torch.equal(got, want), f"replay {k}: tensor {i}"
        eager.forward(X)  # the program's own work between the replays


def test_two_blocks_on_two_streams_at_once():
    n, size, c = 64, 10, 64
    x, dy = _inputs(n, size, c)
    X, DY = dev(x), dev(dy)

    def steps(b):
        for _ in range(3):
            b.forward(X)
            b.backward(X, DY)
            b.step()

    def state(b):
        return (b.y, b.dx, b.dw, b.w, b.momentum, b.gamma, b.beta)

    alone = [two_level_block.Block(n, size, c, seed=k) for k in (1, 2)]
    for b in alone:
        steps(b)
    torch.cuda.synchronize()
    both = [two_level_block.Block(n, size, c, seed=k) for k in (1, 2)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for b, s in zip(both, streams):
        with torch.cuda.stream(s):
            steps(b)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for i, (want, got) in enumerate(zip(state(a), state(b))):
            assert torch.equal(got, want), f"tensor {i}"

"""Layer norm of tensors whose workgroups take several rows or tiles each: the
loops of every kernel (rows held by part of a wave, a wave, several waves, rows
read in turn, tiles of the MX forms), in place too. Bounds are those of
test_gpu_layer_norm.py."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
from gpu_common import dev, host, say
from test_gpu_layer_norm import (_backward, _check_backward, _check_forward, _columns_close, _forward, _inputs, _nan,
                                 _same_codes)

pytestmark = pytest.mark.gpu
EPS32 = float(np.float32(1e-5))  # what the call's fp32 eps holds: 2.5e-8 off 1e-5, more than rstd's last digits where it is most of the variance

# more rows than the workgroups of a launch hold at a time (2048 of 256 threads, 1024 of 512, 512 of 1024 at the most), of
# each way to hold a row: 1 to 64 lanes, two and four quads, 4 and 8 waves, rows read in turn
FP32 = [(25, 41, 640, 3), (80, 80, 16, 64), (3, 1000, 7, 129), (1, 4300, 2, 257), (1, 1300, 7, 700), (1, 1500, 6, 1000),
        (1, 300, 9, 1028), (1, 460, 5, 2048), (1, 433, 5, 4095), (2, 257, 2, 6000), (1, 2100, 1, 4100), (1, 2059, 1, 8193)]


@pytest.mark.parametrize("shape", FP32, ids=str)
def test_rows_of_several_turns(shape):
    x, dy, skip, gamma, beta = _inputs(shape, 3 * sum(shape))
    G, B, X, DY, SK = (dev(t) for t in (gamma, beta, x, dy, skip))
    say(f"layer norm {shape}")
    got = _forward(shape, X, G, B)
    _check_forward(x, gamma, beta, got, eps=EPS32)
    out = _backward(shape, DY, X, G, got[1], got[2], dskip=SK)
    _check_backward(dy, x, gamma, host(got[1]), host(got[2]), skip, out)
    # with a residual, and in place
    say(f"layer norm {shape} in place")
    total, y = X.clone(), SK.clone()
    s = _forward(shape, total, G, B, residual=y, sum=total, y=y)
    assert torch.equal(total, X + SK)
    ref = _forward(shape, total, G, B)
    assert all(torch.equal(a, b) for a, b in zip(s, ref))
    y = X.clone()
    _forward(shape, y, G, B, y=y)
    assert torch.equal(y, got[0])
    for which in range(3):
        t = [DY.clone(), X.clone(), SK.clone()]
        again = _backward(shape, t[0], t[1], G, got[1], got[2], dskip=t[2], dx=t[which])
        assert all(torch.equal(a, b) for a, b in zip(again, out)), which


# more than 2048 tiles of 32 rows: whole pixels, several tiles a pixel, ragged last ones; rows of 16, 32 and 64 lanes; and of
# the two-pass form
MX = [(80, 80, 16, 64), (47, 61, 33, 36), (50, 45, 32, 128), (48, 47, 17, 256), (91, 90, 9, 100), (40, 29, 70, 180),
      (1, 2100, 3, 20), (1, 900, 5, 1000)]


@pytest.mark.parametrize("shape", MX, ids=str)
@pytest.mark.parametrize("fmt", [0, 2, 4])
def test_mx_tiles_of_several_turns(shape, fmt):
    x, dy, skip, gamma, beta = (dev(t) for t in _inputs(shape, 70 + fmt))
    for bp, extra in ((32, True), (1, False)):
        say(f"layer norm mx {shape} fmt={fmt} bp={bp} skip={extra}")
        total = x.clone() if extra else None  # the sum takes the place of x
        y, mean, rstd = _forward(shape, x, gamma, beta, residual=skip if extra else None, sum=_nan(*shape) if extra else None)
        t, mean2, rstd2 = _forward(shape, total if extra else x, gamma, beta, mx=(fmt, bp), residual=skip if extra else None, sum=total)
        assert torch.equal(mean, mean2) and torch.equal(rstd, rstd2) and (not extra or torch.equal(total, x + skip))
        ref = mq.MxTensor.empty(mq.ROLE_ACT, fmt, bp, shape)
        mq.mqconv_quantize(y, ref)
        _same_codes(t, ref, f"y {shape}")
        s = total if extra else x
        dx, _, _ = _backward(shape, dy, s, gamma, mean, rstd, dskip=skip if extra else None)
        t, dg, db = _backward(shape, dy, s, gamma, mean, rstd, mx=(fmt, bp), dskip=skip if extra else None)
        _columns_close(shape, dy, s, mean, rstd, dg, db)
        ref = mq.MxTensor.empty(mq.ROLE_GRAD, fmt, bp, shape)
        mq.mqconv_quantize(dx, ref)
        _same_codes(t, ref, f"dx {shape}")


@pytest.mark.parametrize("shape", [(7, 9, 3, 45), (1, 3, 5, 1024), (1, 1, 3, 20000)], ids=str)
@pytest.mark.parametrize("size", [1e37, 1e-36])
def test_values_near_the_ends_of_the_range(shape, size):
    """x - mean up to 1e38 and rstd of 1e-37; 1e-36 and 1e36, with eps = 0: the ends of what fp32's normal range allows."""
    x, _, _, gamma, beta = _inputs(shape, 15)
    x = (x * np.float32(size)).astype(np.float32)
    got = _forward(shape, dev(x), dev(gamma), dev(beta), eps=0.0)
    _check_forward(x, gamma, beta, got, eps=0.0)

"""MX results of tensors so large that every workgroup walks over several
tiles: the next tile's values are requested ahead, two LDS buffers alternate,
and parameters stay in registers. Bit for bit against the quantization of the
fp32 results. A chip holds at most 1,024 workgroups of eight waves, so these
shapes take three steps and more, the last one not full."""
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
from gpu_common import say, workspace

pytestmark = pytest.mark.gpu
# (H, W, N, C, groups): whole runs of channels with 17 samples, with 3 (several
# pixels a tile), with two tiles along the samples and two slices of channels;
# partial runs
SHAPES = [(121, 119, 17, 64, 16), (301, 299, 3, 64, 8), (61, 59, 33, 320, 32), (111, 109, 17, 72, 9)]
FORMATS = [0, 3, 4]  # runs of 32, 24 and 16 bytes


def _tensors(shape, k):
    h, w, n, c = shape[:4]
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    return [torch.randn(h, w, n, c, generator=g, device="cuda") for _ in range(k)]


def _pair(role, fmt, bp, dims):
    ref, t = (mq.MxTensor.empty(role, fmt, bp, dims) for _ in range(2))
    t.codes.fill_(0xAB)
    t.scales.fill_(0xAB)
    return ref, t


def _same(t, ref, what):
    assert torch.equal(t.scales, ref.scales), what
    assert torch.equal(t.codes, ref.codes), what


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("bp", [1, 32])
def test_norm_and_its_gradient(shape, bp):
    h, w, n, c, g = shape
    x, dy = _tensors(shape, 2)
    gamma, beta = 1 + 0.2 * x[0, 0, 0], 0.3 * dy[0, 0, 0]
    gn = mq.mq_norm(h, w, n, c, g, mq.ACT_SILU)
    drop = mq.mq_drop(0.2, 77)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = (torch.empty(n, g, device="cuda") for _ in range(2))
    ws = workspace(max(mq.mqconv_group_norm_workspace_bytes(gn, k) for k in (0, 1)))
    mq.mqconv_group_norm(gn, x, gamma, beta, y, mean, rstd, ws, drop=drop)
    mq.mqconv_group_norm_backward(gn, dy, x, gamma, beta, mean, rstd, dx, ws=ws, drop=drop)
    for fmt in FORMATS:
        say(f"walk norm {shape} fmt={fmt} bp={bp}")
        ref, t = _pair(mq.ROLE_ACT, fmt, bp, shape[:4])
        mq.mqconv_quantize(y, ref)
        mq.mqconv_group_norm_mx(gn, x, gamma, beta, t, ws=ws, drop=drop)
        _same(t, ref, "y")
        ref, t = _pair(mq.ROLE_GRAD, fmt, bp, shape[:4])
        mq.mqconv_quantize(dx, ref)
        mq.mqconv_group_norm_backward_mx(gn, dy, x, gamma, beta, mean, rstd, t, ws=ws, drop=drop)
        _same(t, ref, "dx")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("bp", [1, 32])
def test_dropout(shape, bp):
    (x,) = _tensors(shape, 1)
    d = mq.mq_drop(0.3, 9)
    y = torch.empty_like(x)
    mq.mqconv_dropout(x, d, y)
    for fmt in FORMATS:
        say(f"walk dropout {shape} fmt={fmt} bp={bp}")
        ref, t = _pair(mq.ROLE_GRAD, fmt, bp, shape[:4])
        mq.mqconv_quantize(y, ref)
        mq.mqconv_dropout_mx(x, d, t)
        _same(t, ref, "dropout")


@pytest.mark.parametrize("shape", [(61, 59, 33, 256), *(s[:4] for s in SHAPES)], ids=str)
@pytest.mark.parametrize("bp", [1, 32])
def test_cache_write_and_read(shape, bp):
    """Stored samples (each as its own quantization in lines) and packed batches read back."""
    h, w, n, c = shape
    (x,) = _tensors(shape, 1)
    order = torch.randperm(n + 2, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32).cuda()
    for fmt in FORMATS:
        say(f"walk cache {shape} fmt={fmt} bp={bp}")
        cache = mq.MxCache.empty(fmt, n + 2, h, w, c)
        mq.mqconv_cache_write(cache, x, order)
        lines = mq.MxTensor.empty(mq.ROLE_ACT, fmt, 1, shape)
        mq.mqconv_quantize(x, lines)
        at = order.long()
        assert torch.equal(cache.codes.view(n + 2, h * w, -1)[at].transpose(0, 1).reshape(-1), lines.codes.view(-1))
        assert torch.equal(cache.scales.view(n + 2, h * w, -1)[at].transpose(0, 1).reshape(-1), lines.scales.view(-1))
        v = torch.empty_like(x)
        mq.mqconv_cache_read(cache, order, v)
        for out in (fmt, 1):
            ref, t = _pair(mq.ROLE_ACT, out, bp, shape)
            mq.mqconv_quantize(v, ref)
            mq.mqconv_cache_read_mx(cache, order, t)
            _same(t, ref, f"read as {out}")

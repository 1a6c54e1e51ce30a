"""The operators around the convolutions on fp32 tensors at any 4-byte address:
bit for bit what they give on tensors that are aligned to whole cache lines."""
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
from gpu_common import say

pytestmark = pytest.mark.gpu
SHAPES = [(16, 16, 4, 32, 8), (5, 3, 33, 45, 9), (64, 48, 6, 64, 16), (57, 61, 17, 33, 11)]


def _at(t, words):
    """A copy of t that starts `words` floats after a 256-byte boundary."""
    buf = torch.empty(t.numel() + 64, dtype=t.dtype, device="cuda")
    v = buf[words:words + t.numel()].view(t.shape)
    assert v.data_ptr() % 256 == 4 * words
    return v.copy_(t)


def _all(shape, words):
    """Every result from inputs and to outputs at that offset, and the floats around the outputs."""
    h, w, n, c, g = shape
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: _at(torch.randn(*s, generator=gen, device="cuda"), words)  # noqa: E731
    x, dy, gamma, beta = r(h, w, n, c), r(h, w, n, c), r(c), r(c)
    outs = []

    def out(*s):
        size = 1
        for d in s:
            size *= d
        buf = torch.full((size + 64,), -7.0, device="cuda")
        outs.append((buf, words, size))
        return buf[words:words + size].view(s)

    gn, drop = mq.mq_norm(h, w, n, c, g, mq.ACT_SILU), mq.mq_drop(0.25, 3)
    ws = torch.empty(max(mq.mqconv_group_norm_workspace_bytes(gn, k) for k in (0, 1)), dtype=torch.uint8, device="cuda")
    mean, rstd = out(n, g), out(n, g)
    mq.mqconv_group_norm(gn, x, gamma, beta, out(h, w, n, c), mean, rstd, ws, drop=drop)
    mq.mqconv_group_norm_backward(gn, dy, x, gamma, beta, mean, rstd, out(h, w, n, c), out(c), out(c), ws, drop=drop)
    mq.mqconv_dropout(x, drop, out(h, w, n, c), residual=dy)
    packed = [mq.MxTensor.empty(role, 0, 32, shape[:4]) for role in (mq.ROLE_ACT, mq.ROLE_GRAD, mq.ROLE_ACT)]
    mq.mqconv_group_norm_mx(gn, x, gamma, beta, packed[0], ws=ws, drop=drop)
    mq.mqconv_group_norm_backward_mx(gn, dy, x, gamma, beta, mean, rstd, packed[1], ws=ws, drop=drop)
    mq.mqconv_dropout_mx(x, drop, packed[2])
    cache = mq.MxCache.empty(3, n, h, w, c)
    slot = _at(torch.arange(n, dtype=torch.int32, device="cuda").flip(0), words)
    mq.mqconv_cache_write(cache, x, slot)
    mq.mqconv_cache_read(cache, slot, out(h, w, n, c))
    torch.cuda.synchronize()
    for i, (buf, at, size) in enumerate(outs):
        assert bool((buf[:at] == -7).all()) and bool((buf[at + size:] == -7).all()), f"output {i} wrote beside itself"
    return [b[a:a + s] for b, a, s in outs] + [t for p in packed for t in (p.codes, p.scales)] + [cache.codes, cache.scales]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_any_4_byte_address(shape):
    ref = _all(shape, 0)
    for words in (1, 2, 3, 5):
        say(f"offset {4 * words} {shape}")
        for i, (a, b) in enumerate(zip(_all(shape, words), ref)):
            assert torch.equal(a, b), f"result {i} at an offset of {4 * words} bytes"

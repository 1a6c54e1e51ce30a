"""The replay cache on the GPU, bit for bit against the oracle's lines:
writing (every format, odd sizes, slots that are out of range or repeated,
parts of a batch), reading as values and as packed activations, empty slots,
non-finite blocks and a cache whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
from oracle import block
from gpu_common import dev, host, say

pytestmark = pytest.mark.gpu
# (H, W, C, slots, samples)
SHAPES = [(1, 1, 1, 1, 1), (1, 1, 64, 9, 5), (3, 5, 45, 7, 4), (20, 20, 256, 12, 6), (7, 1, 300, 5, 5), (9, 11, 33, 4, 2)]


def _slots(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cache(fmt, shape):
    h, w, c, slots, _ = shape
    cache = mq.MxCache.empty(fmt, slots, h, w, c)
    cache.codes.fill_(0xAB)
    cache.scales.fill_(0xAB)
    return cache


def _filled(fmt, shape, seed):
    """A cache with every slot written, and its values."""
    h, w, c, slots, _ = shape
    x = np.random.default_rng(seed).standard_normal((h, w, slots, c)).astype(np.float32)
    cache = _cache(fmt, shape)
    mq.mqconv_cache_write(cache, dev(x), _slots(*range(slots)))
    codes, scales = block.cache_lines(x, fmt)
    return cache, codes, scales, block.cache_values(codes, scales, fmt, h, w, c)


def _rows(cache):
    return host(cache.codes).reshape(cache.slots, -1), host(cache.scales).reshape(cache.slots, -1)


@pytest.mark.parametrize("fmt", range(5))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_write_then_read(fmt, shape):
    say(f"cache {shape} fmt={fmt}")
    h, w, c, slots, n = shape
    rng = np.random.default_rng(fmt)
    x = rng.standard_normal((h, w, n, c)).astype(np.float32)
    order = rng.permutation(slots)[:n]
    cache = _cache(fmt, shape)
    mq.mqconv_cache_write(cache, dev(x), _slots(*order))
    rc, rs = block.cache_lines(x, fmt)
    gc, gs = _rows(cache)
    np.testing.assert_array_equal(gc[order], rc)
    np.testing.assert_array_equal(gs[order], rs)
    rest = np.setdiff1d(np.arange(slots), order)
    assert (gc[rest] == 0xAB).all() and (gs[rest] == 0xAB).all()
    # read back: some slot twice, some slot out of range
    pick = [int(order[0]), int(order[-1]), -1, slots, int(order[0])]
    ref = np.zeros((h, w, len(pick), c), np.float64)
    v = block.cache_values(rc, rs, fmt, h, w, c)
    ref[:, :, [0, 4]] = v[:, :, [0]]
    ref[:, :, 1] = v[:, :, n - 1]
    out = torch.full((h, w, len(pick), c), float("nan"), device="cuda")
    mq.mqconv_cache_read(cache, _slots(*pick), out)
    np.testing.assert_array_equal(host(out), ref.astype(np.float32))


def test_parts_of_a_batch():
    shape = (4, 3, 40, 6, 0)
    x = np.random.default_rng(1).standard_normal((4, 3, 9, 40)).astype(np.float32)
    cache = _cache(0, shape)
    mq.mqconv_cache_write(cache, dev(x), _slots(5, 1), n0=6)
    rc, rs = block.cache_lines(x[:, :, 6:8], 0)
    gc, gs = _rows(cache)
    np.testing.assert_array_equal(gc[[5, 1]], rc)
    np.testing.assert_array_equal(gs[[5, 1]], rs)
    out = torch.full((4, 3, 7, 40), 3.25, device="cuda")
    mq.mqconv_cache_read(cache, _slots(1, 5), out, n0=4)
    v = block.cache_values(rc, rs, 0, 4, 3, 40).astype(np.float32)
    got = host(out)
    np.testing.assert_array_equal(got[:, :, 4:6], v[:, :, ::-1])
    assert (got[:, :, :4] == 3.25).all() and (got[:, :, 6:] == 3.25).all()


def test_the_last_of_several_samples_with_one_slot_is_stored():
    n = 700
    x = np.random.default_rng(2).standard_normal((2, 2, n, 32)).astype(np.float32)
    slot = np.random.default_rng(3).integers(-2, 12, n).astype(np.int32)  # ten slots, some numbers out of range
    cache = _cache(4, (2, 2, 32, 10, n))
    mq.mqconv_cache_write(cache, dev(x), dev(slot))
    last = [int(np.flatnonzero(slot == s)[-1]) for s in range(10)]
    rc, rs = block.cache_lines(x[:, :, last], 4)
    gc, gs = _rows(cache)
    np.testing.assert_array_equal(gc, rc)
    np.testing.assert_array_equal(gs, rs)


def test_every_slot_out_of_range_writes_nothing():
    cache = _cache(2, (3, 3, 33, 4, 3))
    mq.mqconv_cache_write(cache, dev(np.ones((3, 3, 3, 33), np.float32)), _slots(-1, 4, 2**31 - 1))
    assert (host(cache.codes) == 0xAB).all() and (host(cache.scales) == 0xAB).all()


@pytest.mark.parametrize("fmt", range(5))
def test_special_values(fmt):
    """Zeros of both signs, subnormals, saturation, non-finite blocks."""
    rng = np.random.default_rng(60 + fmt)
    x = rng.standard_normal((4, 2, 3, 64)).astype(np.float32)
    x[0, 0] = 0.0
    x[0, 1] = -0.0
    x[1, 0] = np.float32(2.0 ** -130) * rng.choice([-1, 1], (3, 64))
    x[1, 1] = np.float32(3e38) * rng.uniform(-1, 1, (3, 64)).astype(np.float32)
    x[2, 0, 1, 5] = np.nan
    x[2, 1, 2, 40] = np.inf
    x[3, 0] = rng.choice([-1.0, 1.0], (3, 64)) * rng.integers(0, 64, (3, 64)) / 8.0
    cache = _cache(fmt, (4, 2, 64, 3, 3))
    mq.mqconv_cache_write(cache, dev(x), _slots(0, 1, 2))
    rc, rs = block.cache_lines(x, fmt)
    gc, gs = _rows(cache)
    np.testing.assert_array_equal(gc, rc)
    np.testing.assert_array_equal(gs, rs)
    out = torch.empty((4, 2, 3, 64), device="cuda")
    mq.mqconv_cache_read(cache, _slots(0, 1, 2), out)
    v = block.cache_values(rc, rs, fmt, 4, 2, 64)
    got = host(out)
    nan = np.isnan(v)
    assert nan.sum() == 2 * 32 and np.array_equal(np.isnan(got), nan)
    np.testing.assert_array_equal(got[~nan], v[~nan].astype(np.float32))
    assert np.array_equal(np.signbit(got[~nan]), np.signbit(v[~nan]))


@pytest.mark.parametrize("fmt", range(5))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_read_mx_is_the_quantized_read(fmt, shape):
    h, w, c, slots, _ = shape
    cache, codes, scales, _ = _filled(fmt, shape, 70 + fmt)
    for n in (1, 3, 16, 33):
        slot = np.random.default_rng(n).integers(-1, slots + 1, n).astype(np.int32)
        x = torch.empty((h, w, n, c), device="cuda")
        mq.mqconv_cache_read(cache, dev(slot), x)
        for out in range(5):
            for bp in (1, 32):
                say(f"cache read_mx {shape} n={n} {fmt} -> {out} bp={bp}")
                ref, t = (mq.MxTensor.empty(mq.ROLE_ACT, out, bp, (h, w, n, c)) for _ in range(2))
                mq.mqconv_quantize(x, ref)
                t.codes.fill_(0xAB)
                t.scales.fill_(0xAB)
                mq.mqconv_cache_read_mx(cache, dev(slot), t)
                np.testing.assert_array_equal(host(t.scales), host(ref.scales))
                np.testing.assert_array_equal(host(t.codes), host(ref.codes))
                if out == fmt and bp == 1:  # stored codes come back unchanged
                    ok = (slot >= 0) & (slot < slots)
                    got = host(t.codes).reshape(h * w, n, -1)[:, ok].transpose(1, 0, 2).reshape(ok.sum(), codes.shape[1])
                    np.testing.assert_array_equal(got, codes[slot[ok]])


def test_read_mx_of_non_finite_blocks():
    x = np.random.default_rng(5).standard_normal((2, 2, 3, 64)).astype(np.float32)
    x[0, 1, 1, 3] = np.nan
    cache = _cache(0, (2, 2, 64, 3, 3))
    mq.mqconv_cache_write(cache, dev(x), _slots(0, 1, 2))
    v = torch.empty((2, 2, 3, 64), device="cuda")
    mq.mqconv_cache_read(cache, _slots(0, 1, 2), v)
    for bp in (1, 32):
        ref, t = (mq.MxTensor.empty(mq.ROLE_ACT, 3, bp, (2, 2, 3, 64)) for _ in range(2))
        mq.mqconv_quantize(v, ref)
        mq.mqconv_cache_read_mx(cache, _slots(0, 1, 2), t)
        np.testing.assert_array_equal(host(t.scales), host(ref.scales))
        np.testing.assert_array_equal(host(t.codes), host(ref.codes))
        assert (host(t.scales) == 255).sum() == 1


def test_offsets_beyond_32_bits():
    """5,000 slots of 1 MiB of codes: the last slots lie beyond 4 GiB."""
    h, w, c, slots = 32, 32, 1024, 5000
    say("cache beyond 32 bits")
    cache = mq.MxCache.empty(0, slots, h, w, c)
    assert cache.codes.numel() > 2**32
    x = torch.randn((h, w, 3, c), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    mq.mqconv_cache_write(cache, x, _slots(slots - 1, 4097, 0))
    out, q, ref = torch.empty_like(x), *(mq.MxTensor.empty(mq.ROLE_ACT, 0, 1, (h, w, 3, c)) for _ in range(2))
    mq.mqconv_cache_read(cache, _slots(slots - 1, 4097, 0), out)
    mq.mqconv_quantize(x, ref)
    mq.mqconv_cache_read_mx(cache, _slots(slots - 1, 4097, 0), q)
    assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)
    back = mq.MxTensor.empty(mq.ROLE_ACT, 0, 1, (h, w, 3, c))
    mq.mqconv_quantize(out, back)
    assert torch.equal(back.codes, ref.codes)


def test_another_stream_and_graph():
    h, w, c, slots = 5, 4, 70, 6
    cache = _cache(3, (h, w, c, slots, 0))
    x = dev(np.random.default_rng(8).standard_normal((h, w, 4, c)).astype(np.float32))
    to, at = _slots(5, 2, 0, 3), _slots(3, 3, 2, 1, 5)
    out = torch.empty((h, w, 5, c), device="cuda")
    q = mq.MxTensor.empty(mq.ROLE_ACT, 1, 32, (h, w, 5, c))
    cache.codes.zero_()
    cache.scales.fill_(120)

    def path():
        mq.mqconv_cache_write(cache, x, to)
        mq.mqconv_cache_read(cache, at, out)
        mq.mqconv_cache_read_mx(cache, at, q)

    path()
    eager = [t.clone() for t in (cache.codes, cache.scales, out, q.codes, q.scales)]
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        path()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            path()
    torch.cuda.synchronize()
    for _ in range(4):
        for t in (out, q.codes, q.scales):
            t.fill_(1)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        for t, e in zip((cache.codes, cache.scales, out, q.codes, q.scales), eager):
            assert torch.equal(t, e)
        path()

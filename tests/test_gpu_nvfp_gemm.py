"""The three products on two-level codes on the GPU, against the oracle's direct
convolutions (fp64) of its own quantization of the same tensors.

Bound, with S the sum of an output's absolute products and e = 2^-24: products
are exact. The matrix units add 16 products to an accumulator at a time, dropping
at most 2^-26 of the largest of the 17 for each of the 16 (2^-22 of S) and
rounding once (e S); with k products that happens k' / 16 times, k' the extent
of the sum with its padding (channels to 64; samples to 8, their pixels to 64).
Slices of a sum are added with one rounding each (at most 64), and three
roundings apply the tensors' scales, themselves rounded twice:
  |y - y'| <= ((2^-22 + e) k' / 16 + 64 e [slices]) S + 5 e |y| + 2^-149,
the last for results below fp32's normal range, where values are 2^-149 apart
and a rounding is off by up to half of that whatever the value."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
import oracle
from gpu_common import dev, host, say, workspace

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
up = lambda v, m: -(-v // m) * m  # noqa: E731

# (n, cin, h, w, cout, kh, kw, sh, sw, ph, pw)
LINEAR = [(n, cin, 1, 1, cout, 1, 1, 1, 1, 0, 0) for n, cin, cout in
          ((1, 1, 1), (1, 64, 64), (1, 300, 70), (2, 45, 9), (3, 200, 130), (5, 1030, 33), (8, 64, 257), (9, 33, 65), (16, 1024, 64),
           (17, 130, 70), (31, 64, 100), (64, 512, 64), (130, 96, 140), (300, 200, 130), (1000, 72, 300))]
CONVS = [
    (2, 32, 16, 16, 32, 3, 3, 1, 1, 1, 1), (1, 3, 13, 17, 16, 3, 3, 2, 2, 1, 1), (5, 45, 19, 23, 90, 3, 3, 2, 2, 1, 1),
    (16, 64, 10, 11, 64, 3, 3, 1, 1, 1, 1), (33, 40, 9, 10, 36, 3, 3, 2, 2, 1, 1), (7, 70, 5, 4, 33, 5, 3, 1, 2, 2, 0),
    (4, 8, 15, 16, 8, 15, 15, 1, 1, 7, 7), (9, 16, 12, 11, 24, 1, 1, 2, 2, 0, 0), (2, 130, 7, 9, 257, 2, 2, 3, 1, 1, 0),
    (3, 24, 9, 9, 40, 2, 1, 8, 5, 0, 0), (64, 72, 6, 5, 136, 3, 3, 1, 1, 1, 1), (128, 64, 4, 4, 32, 3, 3, 2, 1, 1, 1),
    (12, 20, 1, 40, 30, 1, 3, 1, 1, 0, 1), (16, 8, 60, 60, 64, 3, 3, 1, 1, 1, 1),
]
# rows enough for the kernel that reads the codes itself: one and two tiles of columns, ragged ones, channels that end inside a
# run and inside a block, strides (and pixels that no tap reaches), samples that end inside a block, sums in slices, a linear layer
CODES = [
    (16, 64, 16, 16, 64, 3, 3, 1, 1, 1, 1), (5, 32, 30, 30, 100, 3, 3, 1, 1, 1, 1), (20, 96, 33, 31, 160, 3, 3, 2, 2, 1, 1),
    (64, 250, 9, 9, 64, 3, 3, 1, 1, 1, 1), (4100, 320, 1, 1, 70, 1, 1, 1, 1, 0, 0), (7, 58, 40, 39, 30, 5, 3, 1, 2, 2, 0),
    (9, 27, 60, 61, 32, 1, 1, 2, 2, 0, 0), (33, 128, 23, 24, 224, 2, 2, 3, 1, 1, 0),
]
# more tiles than the chip holds workgroups, which then take several: whole tiles, and a last one that is not
MANY_TILES = [(64, 32, 64, 64, 96, 3, 3, 1, 1, 1, 1), (65, 96, 63, 65, 32, 3, 3, 1, 1, 1, 1), (64, 32, 64, 64, 64, 1, 1, 1, 1, 0, 0)]
OPS = ("forward", "data", "weight")


def _inputs(s, seed, spread=True):
    n, cin, h, w, cout, kh, kw, sh, sw, ph, pw = s
    ho, wo = (h + 2 * ph - kh) // sh + 1, (w + 2 * pw - kw) // sw + 1
    rng = np.random.default_rng(seed)
    wide = lambda *d: np.exp(rng.uniform(-2, 2, size=d[:-1] + (1,))) if spread else 1.0  # noqa: E731
    x = rng.standard_normal((h, w, n, cin)) * wide(h, w, n, cin)
    wt = rng.standard_normal((cout, kh, kw, cin)) * wide(cout, kh, kw, cin)
    dy = 1e-3 * rng.standard_normal((ho, wo, n, cout)) * wide(ho, wo, n, cout)
    return tuple(t.astype(np.float32) for t in (x, wt, dy))


def _quantized(t, role, fmt):
    """On the GPU, and the oracle's values."""
    q = mq.NvfpTensor.empty(role, fmt, t.shape)
    q.quantize(dev(t), workspace(mq.mqconv_nvfp_workspace_bytes()))
    return q, oracle.nvfp_dequantize(role, fmt, *oracle.nvfp_quantize(role, fmt, t))


class _Shape:
    def __init__(self, s):
        self.t = s

    def as_tuple(self):
        return self.t


def _call(s, op, a, b, out=None, fill=0xFF, stream=None):
    fn = (mq.mqconv_nvfp_forward, mq.mqconv_nvfp_backward_data, mq.mqconv_nvfp_backward_weight)[op]
    n, cin, h, w, cout, kh, kw, sh, sw, ph, pw = s
    ho, wo = (h + 2 * ph - kh) // sh + 1, (w + 2 * pw - kw) // sw + 1
    shape = ((ho, wo, n, cout), (h, w, n, cin), (cout, kh, kw, cin))[op]
    if out is None:
        out = torch.full(shape, float("nan"), device="cuda")
    ws = workspace(mq.mqconv_nvfp_gemm_workspace_bytes(s, op, a.fmt, b.fmt)).fill_(fill)
    fn(s, a, b, out, ws, stream=stream)
    return out


def _sum_extent(s, op):
    n, cin, h, w, cout, kh, kw, sh, sw, ph, pw = s
    ho, wo = (h + 2 * ph - kh) // sh + 1, (w + 2 * pw - kw) // sw + 1
    if op == 0:
        return kh * kw * up(cin, 64)
    return -(-kh // sh) * -(-kw // sw) * up(cout, 64) if op == 1 else up(ho * wo * up(n, 8), 64)


def _reference(s, op, a, b):
    if s[2] == s[3] == s[5] == s[6] == 1:  # linear: the same sums as matrix products
        if op == 0:
            return a[0, 0] @ b[:, 0, 0].T
        return a[0, 0] @ b[:, 0, 0] if op == 1 else a[0, 0].T @ b[0, 0]
    return (oracle.conv_fwd, oracle.conv_dgrad, oracle.conv_wgrad)[op](_Shape(s), a, b)


def _close(s, op, got, a, b, label):
    ref = np.asarray(_reference(s, op, a, b)).reshape(got.shape)
    total = np.asarray(_reference(s, op, np.abs(a), np.abs(b))).reshape(got.shape)
    tol = ((2.0 ** -22 + E) * _sum_extent(s, op) / 16 + 64 * E) * total + 5 * E * np.abs(ref) + 2.0 ** -149
    err = np.abs(got.astype(np.float64) - ref)
    say(f"  {OPS[op]} {s} {label}: {np.linalg.norm(err) / max(np.linalg.norm(ref), 1e-300):.2e} relative, "
        f"{(err / np.maximum(tol, 1e-300)).max():.3f} of the bound")
    bad = ~(err <= tol)
    assert not bad.any(), f"{OPS[op]} {s} {label}: {bad.sum()} of {bad.size}, first at {tuple(np.argwhere(bad)[0])}: {got[bad][0]!r} for {ref[bad][0]!r}"


def _operands(s, fx, fw, fdy, seed):
    x, w, dy = _inputs(s, seed)
    X, W, DY = _quantized(x, mq.ROLE_ACT, fx), _quantized(w, mq.ROLE_WEIGHT, fw), _quantized(dy, mq.ROLE_GRAD, fdy)
    return (X, W), (DY, W), (DY, X)


@pytest.mark.parametrize("s", LINEAR + CONVS, ids=lambda s: "x".join(map(str, s)))
def test_products_of_four_bit_codes(s):
    for op, (a, b) in enumerate(_operands(s, 4, 4, 4, sum(s))):
        _close(s, op, host(_call(s, op, a[0], b[0])), a[1], b[1], "e2m1")


@pytest.mark.parametrize("s", CODES + MANY_TILES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fmts", [(4, 4, 4), (0, 4, 1), (1, 2, 0)])
def test_products_from_codes(s, fmts):
    for op, (a, b) in enumerate(_operands(s, *fmts, seed=200 + sum(s))):
        if op < 2:
            _close(s, op, host(_call(s, op, a[0], b[0])), a[1], b[1], str(fmts))


@pytest.mark.parametrize("s", [LINEAR[2], LINEAR[5], LINEAR[13], CONVS[2], CONVS[5], CONVS[10]], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fmts", [(0, 0, 1), (1, 2, 3), (2, 3, 0), (3, 4, 2), (4, 1, 4), (4, 0, 1)])
def test_products_of_every_format(s, fmts):
    for op, (a, b) in enumerate(_operands(s, *fmts, seed=100 + sum(s))):
        _close(s, op, host(_call(s, op, a[0], b[0])), a[1], b[1], str(fmts))


@pytest.mark.parametrize("s", [(3400, 70, 1, 1, 4096, 1, 1, 1, 1, 0, 0), (256, 4000, 1, 1, 40, 1, 1, 1, 1, 0, 0)], ids=str)
def test_large_linear_layers(s):
    """The largest tiles, and long sums of few outputs."""
    for op, (a, b) in enumerate(_operands(s, 4, 4, 4, 9)):
        _close(s, op, host(_call(s, op, a[0], b[0])), a[1], b[1], "large")


def test_exact_sums():
    """Small whole numbers of one scale have no rounding at all."""
    s = (40, 96, 7, 6, 72, 3, 3, 1, 1, 1, 1)
    rng = np.random.default_rng(1)
    pick = lambda *d: rng.choice(np.float32([-6, -4, -3, -2, -1.5, -1, -0.5, 0, 0.5, 1, 1.5, 2, 3, 4, 6]), size=d)  # noqa: E731
    x, w, dy = pick(7, 6, 40, 96) * 448, pick(72, 3, 3, 96) * 448, pick(7, 6, 40, 72) * 448
    for t, step in ((x, 8), (w, 8), (dy, 8)):
        t[..., ::8] = np.sign(t[..., ::8] + 0.25) * 6 * 448  # every block's largest
    X, W, DY = _quantized(x, 0, 4), _quantized(w, 1, 4), _quantized(dy, 2, 4)
    assert np.array_equal(X[1], x) and np.array_equal(W[1], w) and np.array_equal(DY[1], dy)
    for op, (a, b) in enumerate(((X, W), (DY, W), (DY, X))):
        ref = np.asarray(_reference(s, op, a[1], b[1]))
        assert np.abs(ref).max() / 448 ** 2 * 4 < 2 ** 24
        np.testing.assert_array_equal(host(_call(s, op, a[0], b[0])).astype(np.float64), ref.reshape(host(_call(s, op, a[0], b[0])).shape))


@pytest.mark.parametrize("s", [LINEAR[2], LINEAR[11], CONVS[2]], ids=lambda s: "x".join(map(str, s)))
def test_scales_of_any_size(s):
    """T T' leaves fp32's range where its factors or the result do not."""
    x, w, dy = _inputs(s, 5, spread=False)
    for sx, sw in ((1e30, 1e-30), (1e-30, 1e30), (1e-18, 1e-18), (1e18, 1e16)):
        X, W, DY = _quantized(x * np.float32(sx), 0, 4), _quantized(w * np.float32(sw), 1, 4), _quantized(dy * np.float32(sx), 2, 4)
        XW = _quantized(x * np.float32(sw), 0, 4)
        for op, (a, b) in enumerate(((X, W), (DY, W), (DY, XW))):
            _close(s, op, host(_call(s, op, a[0], b[0])), a[1], b[1], f"{sx} {sw}")


@pytest.mark.parametrize("s", [LINEAR[4], LINEAR[13], CONVS[2], CONVS[10], CODES[1], CODES[5]], ids=lambda s: "x".join(map(str, s)))
def test_nan_blocks_reach_their_outputs_alone_and_zeros_give_zeros(s):
    x, w, dy = _inputs(s, 6)
    W, DY = _quantized(w, 1, 4), _quantized(dy, 2, 4)
    clean = _quantized(x, 0, 4)
    bad = x.copy()
    bad[0, -1, -1, -1] = np.inf  # its block: the last samples' and channels', not whole where these are no multiples of 8
    B = _quantized(bad, 0, 4)
    n0, c0 = (s[0] - 1) // 8 * 8, (s[1] - 1) // 8 * 8
    reach = np.zeros(x.shape)
    reach[0, -1, n0:, c0:] = 1
    assert np.array_equal(np.isnan(B[1]), reach == 1)
    for op, (a, b) in ((0, (B, W)), (2, (DY, B))):
        ref = host(_call(s, op, clean[0] if op == 0 else DY[0], W[0] if op == 0 else clean[0]))
        got = host(_call(s, op, a[0], b[0]))
        # an output is NaN where any of its products, zeros among them, has the block's values
        hit = _reference(s, op, reach, np.ones(w.shape)) if op == 0 else _reference(s, op, np.ones(dy.shape), reach)
        hit = np.asarray(hit).reshape(got.shape) > 0
        assert np.array_equal(np.isnan(got), hit) and hit.any()
        np.testing.assert_allclose(got[~hit], ref[~hit], rtol=0, atol=np.abs(ref).max() * 1e-2)
    Z = _quantized(np.zeros_like(x), 0, 4)
    assert not host(_call(s, 0, Z[0], W[0])).any() and not host(_call(s, 2, DY[0], Z[0])).any()


@pytest.mark.parametrize("s", [LINEAR[2], LINEAR[5], LINEAR[13], CONVS[4], CONVS[2], CODES[1], CODES[3]], ids=lambda s: "x".join(map(str, s)))
def test_repeats_strange_addresses_another_stream_and_guards(s):
    for op, (a, b) in enumerate(_operands(s, 4, 4, 4, 77)):
        a, b = a[0], b[0]
        ref = _call(s, op, a, b)
        for fill in (0, 0x7F):
            assert torch.equal(_call(s, op, a, b, fill=fill), ref)
        big = torch.full((ref.numel() + 9,), 7.0, device="cuda")
        view = big[3:3 + ref.numel()]
        scales = torch.full((b.scales.numel() + 1,), 0x7F, dtype=torch.uint8, device="cuda")  # E4M3 bytes at any address
        scales[1:] = b.scales
        moved = mq.NvfpTensor(b.codes, scales[1:], b.tensor_scale, b.fmt, b.role, b.dims)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        ws = workspace(mq.mqconv_nvfp_gemm_workspace_bytes(s, op, 4, 4))
        (mq.mqconv_nvfp_forward, mq.mqconv_nvfp_backward_data, mq.mqconv_nvfp_backward_weight)[op](s, a, moved, view, ws, stream=st)
        st.synchronize()
        assert torch.equal(view, ref.reshape(-1)) and (big[:3] == 7).all() and (big[3 + ref.numel():] == 7).all()


@pytest.mark.parametrize("s", [LINEAR[2], LINEAR[13], CONVS[2], CODES[3]], ids=lambda s: "x".join(map(str, s)))
def test_graph_replays_are_the_eager_results(s):
    first, second = _operands(s, 4, 4, 4, 41), _operands(s, 4, 4, 4, 42)
    used = [[_clone(t[0]) for t in pair] for pair in first]
    outs = [_call(s, op, *pair) for op, pair in enumerate(used)]
    wss = [workspace(mq.mqconv_nvfp_gemm_workspace_bytes(s, op, 4, 4)) for op in range(3)]
    fns = (mq.mqconv_nvfp_forward, mq.mqconv_nvfp_backward_data, mq.mqconv_nvfp_backward_weight)

    def path():
        for fn, pair, out, ws in zip(fns, used, outs, wss):
            fn(s, *pair, out, ws)

    def load(which):
        for pair, new in zip(used, which):
            for t, v in zip(pair, new):
                for k in ("codes", "scales", "tensor_scale"):
                    getattr(t, k).copy_(getattr(v[0], k))

    eager = []
    for which in (first, second):
        load(which)
        path()
        eager.append([t.clone() for t in outs])
    assert not torch.equal(eager[0][0], eager[1][0])
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        path()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            path()
    for k in (0, 1, 1, 0):
        load((first, second)[k])
        for t in outs + wss:
            t.fill_(0x5A if t.dtype == torch.uint8 else float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        for t, e in zip(outs, eager[k]):
            assert torch.equal(t, e)
        path()


def _clone(t):
    return mq.NvfpTensor(t.codes.clone(), t.scales.clone(), t.tensor_scale.clone(), t.fmt, t.role, t.dims)


def test_injected_failures_then_recovery():
    s = CONVS[2]
    for op, (a, b) in enumerate(_operands(s, 4, 4, 4, 3)):
        ref = _call(s, op, a[0], b[0])
        failed = 0
        try:
            for k in range(1, 12):
                mq.mqconv_inject_launch_failure(k)
                try:
                    got = _call(s, op, a[0], b[0])
                except mq.MqConvError as e:
                    assert e.status == -7
                    failed += 1
                    continue
                mq.mqconv_inject_launch_failure(0)
                assert torch.equal(got, ref)
                break
            else:
                pytest.fail("every call failed")
        finally:
            mq.mqconv_inject_launch_failure(0)
        assert failed >= 2


@pytest.mark.parametrize("fmts", [(4, 4), (0, 0), (1, 1), (2, 2), (3, 3), (0, 4), (2, 1)], ids=str)
def test_few_rows_of_many_channels(fmts):
    """Channels shared by 1, 2 and 4 waves, and more than those hold at once; single rows of two formats."""
    for n, cin, cout in ((1, 2048, 9), (1, 2049, 70), (2, 4100, 33), (3, 7000, 8), (8, 9000, 50), (5, 20000, 5), (1, 40009, 3)):
        if n > 1 and fmts[0] != fmts[1] and cin > 5000:
            continue
        s = (n, cin, 1, 1, cout, 1, 1, 1, 1, 0, 0)
        x, w, _ = _inputs(s, 90 + n)
        X, W = _quantized(x, mq.ROLE_ACT, fmts[0]), _quantized(w, mq.ROLE_WEIGHT, fmts[1])
        first = _call(s, 0, X[0], W[0])
        _close(s, 0, host(first), X[1], W[1], str(fmts))
        assert torch.equal(_call(s, 0, X[0], W[0], fill=0), first)

"""Products of two-level codes on the ways through their kernels that small
tensors do not take: workgroups that take several whole tiles of every width
(whose first loads are waited for with the stores of the tile before under
way), the largest tiles with several taps, NaN blocks in every kind of operand,
and block scales at any address.

Large results are compared with fp64 products of the oracle's values, tap by
tap on the GPU (their own error, 2^-53 a term, disappears in the bound), under
the bound of test_gpu_nvfp_gemm.py:
  |y - y'| <= ((2^-22 + e) k' / 16 + 64 e) S + 5 e |y| + 2^-149."""
import numpy as np
import pytest
import torch

import microscaling_quantized_convolution_mxq_amd as mq
from gpu_common import host, say, workspace
from test_gpu_nvfp_gemm import CODES, E, LINEAR, MANY_TILES, OPS, _call, _close, _inputs, _operands, _quantized, _reference, _sum_extent

pytestmark = pytest.mark.gpu
FNS = (mq.mqconv_nvfp_forward, mq.mqconv_nvfp_backward_data, mq.mqconv_nvfp_backward_weight)


def _product64(s, op, a, b):
    """Forward product or input gradient in fp64, a tap at a time."""
    n, cin, h, w, cout, kh, kw, sh, sw, ph, pw = s
    ho, wo = (h + 2 * ph - kh) // sh + 1, (w + 2 * pw - kw) // sw + 1
    padded = torch.zeros(h + 2 * ph, w + 2 * pw, n, cin, dtype=torch.float64, device="cuda")
    if op == 0:
        padded[ph:ph + h, pw:pw + w] = a
    out = torch.zeros(ho * wo * n, cout, dtype=torch.float64, device="cuda")
    for i in range(kh):
        for j in range(kw):
            tap = (slice(i, i + sh * (ho - 1) + 1, sh), slice(j, j + sw * (wo - 1) + 1, sw))
            if op == 0:
                out += padded[tap].reshape(-1, cin) @ b[:, i, j].t()
            else:
                padded[tap] += (a.reshape(-1, cout) @ b[:, i, j]).view(ho, wo, n, cin)
    return out.view(ho, wo, n, cout) if op == 0 else padded[ph:ph + h, pw:pw + w]


def _check(s, op, a, b, label):
    """a, b: (codes, the oracle's values) of the operands."""
    got = _call(s, op, a[0], b[0]).double()
    A, B = (torch.from_numpy(np.asarray(v, np.float64)).cuda() for v in (a[1], b[1]))
    ref, total = _product64(s, op, A, B), _product64(s, op, A.abs(), B.abs())
    tol = ((2.0 ** -22 + E) * _sum_extent(s, op) / 16 + 64 * E) * total + 5 * E * ref.abs() + 2.0 ** -149
    err = (got - ref).abs()
    say(f"  {OPS[op]} {s} {label}: {float(err.norm() / ref.norm()):.2e} relative, {float((err / tol).max()):.3f} of the bound")
    bad = ~(err <= tol)
    assert not bad.any(), f"{OPS[op]} {s} {label}: {int(bad.sum())} of {bad.numel()}, first at {tuple(bad.nonzero()[0].tolist())}"


# Tiles whose columns are all there (64, 128, 2 x 128), more of them than the chip holds workgroups, sums of several steps:
# (shape, op, steps of a sum, whole tiles of rows or a last one that is not).
WHOLE = [
    ((64, 64, 64, 64, 64, 3, 3, 1, 1, 1, 1), 0), ((63, 64, 61, 63, 128, 3, 3, 1, 1, 1, 1), 0),
    ((32, 32, 64, 64, 256, 3, 3, 1, 1, 1, 1), 0), ((63, 64, 61, 63, 128, 3, 3, 1, 1, 1, 1), 1),
    ((64, 128, 64, 64, 96, 3, 3, 2, 2, 1, 1), 1), ((66, 128, 63, 65, 64, 5, 3, 1, 2, 2, 1), 1),
]


@pytest.mark.parametrize("s,op", WHOLE, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else OPS[v])
@pytest.mark.parametrize("fa,fb", [(4, 4), (0, 1), (1, 4), (4, 2)])
def test_many_whole_tiles_from_codes(s, op, fa, fb):
    x, w, dy = _inputs(s, 300 + sum(s))
    a = _quantized(x, mq.ROLE_ACT, fa) if op == 0 else _quantized(dy, mq.ROLE_GRAD, fa)
    _check(s, op, a, _quantized(w, mq.ROLE_WEIGHT, fb), f"{fa} by {fb}")


# 256 x 256 tiles, whose loop asks for steps behind the last tap: one and several blocks of channels, strides, ragged rows and columns
LARGE = [((31, 72, 41, 39, 520, 3, 3, 1, 1, 1, 1), 0), ((31, 520, 41, 39, 72, 3, 3, 2, 2, 1, 1), 1),
         ((40, 24, 37, 36, 300, 2, 3, 1, 1, 1, 0), 0), ((33, 270, 40, 41, 40, 1, 2, 1, 1, 0, 1), 1)]


@pytest.mark.parametrize("s,op", LARGE, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else OPS[v])
@pytest.mark.parametrize("fa,fb", [(4, 4), (2, 1)])
def test_largest_tiles_of_several_taps(s, op, fa, fb):
    x, w, dy = _inputs(s, 400 + sum(s))
    a = _quantized(x, mq.ROLE_ACT, fa) if op == 0 else _quantized(dy, mq.ROLE_GRAD, fa)
    _check(s, op, a, _quantized(w, mq.ROLE_WEIGHT, fb), f"{fa} by {fb}")


# Sums in slices together with classes of rows: four classes of 1 to 4 taps, nine of them (two launches), some that no tap
# reaches; the largest tiles in slices; all from codes and from 16-bit values
SLICED = [((8, 64, 25, 27, 512, 3, 3, 2, 2, 1, 1), 1), ((8, 64, 26, 25, 320, 5, 5, 3, 3, 2, 1), 1),
          ((8, 64, 26, 25, 1024, 2, 2, 3, 3, 1, 1), 1), ((9, 130, 22, 23, 600, 3, 2, 8, 1, 0, 1), 1),
          ((32, 256, 40, 40, 256, 3, 3, 1, 1, 1, 1), 0)]


@pytest.mark.parametrize("s,op", SLICED, ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else OPS[v])
@pytest.mark.parametrize("fa,fb", [(4, 4), (0, 1), (2, 4)])
def test_slices_of_classes_and_of_large_tiles(s, op, fa, fb):
    x, w, dy = _inputs(s, 600 + sum(s))
    a = _quantized(x, mq.ROLE_ACT, fa) if op == 0 else _quantized(dy, mq.ROLE_GRAD, fa)
    _check(s, op, a, _quantized(w, mq.ROLE_WEIGHT, fb), f"{fa} by {fb}")


@pytest.mark.parametrize("n,cin,cout", [(20, 40, 52000), (300, 64, 51300), (3, 5, 60001)])
def test_weight_gradient_of_many_outputs(n, cin, cout):
    """Tall tiles: few columns of dW and tens of thousands of rows."""
    s = (n, cin, 1, 1, cout, 1, 1, 1, 1, 0, 0)
    x, _, dy = _inputs(s, n)
    a, b = _quantized(dy, mq.ROLE_GRAD, 4), _quantized(x, mq.ROLE_ACT, 1)
    _close(s, 2, host(_call(s, 2, a[0], b[0])), a[1], b[1], "tall")


@pytest.mark.parametrize("s", [LINEAR[2], LINEAR[5], LINEAR[13], CODES[1], CODES[5]], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fx,fw", [(0, 0), (1, 4), (4, 1), (0, 2), (3, 3)])
def test_nan_blocks_of_every_format(s, fx, fw):
    """A NaN block of either operand makes the outputs NaN that have one of its values. Outputs that pair such a value with
    zero padding alone (borders under a weight's outer taps, a weight's taps that lead out of the image) are left open by the
    definition; all others are within the bound."""
    x, w, dy = _inputs(s, 7)
    X, W, DY = _quantized(x, mq.ROLE_ACT, fx), _quantized(w, mq.ROLE_WEIGHT, fw), _quantized(dy, mq.ROLE_GRAD, fx)

    def spoilt(t, at, role, fmt):
        """t with an infinity at `at`; its values with zeros for its block's, and where that is (blocks end with the tensor)."""
        t = t.copy()
        t[at] = np.inf
        codes, values = _quantized(t, role, fmt)
        reach = np.isnan(values)
        assert 1 <= reach.sum() <= 64
        return (codes, np.where(reach, 0, values)), reach.astype(np.float64)

    bx, rx = spoilt(x, (0, -1, -1, -1), mq.ROLE_ACT, fx)
    bw, rw = spoilt(w, (-1, 0, 0, -1), mq.ROLE_WEIGHT, fw)
    bd, rd = spoilt(dy, (-1, 0, 0, -1), mq.ROLE_GRAD, fx)
    one = lambda t: np.ones(t.shape)  # noqa: E731
    n, cin, h, w_, cout, kh, kw, sh, sw, ph, pw = s
    # where padding may stand in a product with the block: the weight's tap (0, 0) at every pixel that it can reach from inside
    # or outside the image, a gradient's pixel under every tap
    open_y = np.broadcast_to(rw.any(axis=(1, 2, 3)), dy.shape)
    taps = np.outer((np.arange(h) + ph) % sh == 0, (np.arange(w_) + pw) % sw == 0)
    open_x = np.broadcast_to(taps[:, :, None, None] & rw.any(axis=(0, 1, 2)), x.shape)
    open_w = np.broadcast_to(rd.any(axis=(0, 1, 2))[:, None, None, None], w.shape)
    for op, a, b, ra, rb, left in ((0, bx, W, rx, one(w), None), (0, X, bw, one(x), rw, open_y), (1, bd, W, rd, one(w), None),
                                   (1, DY, bw, one(dy), rw, open_x), (2, DY, bx, one(dy), rx, None), (2, bd, X, rd, one(x), open_w)):
        got = host(_call(s, op, a[0], b[0]))
        hit = np.asarray(_reference(s, op, ra, rb)).reshape(got.shape) > 0
        clean = ~hit if left is None else ~(hit | left)
        label = f"{OPS[op]} {s} {fx} {fw}"
        assert hit.any() and np.isnan(got[hit]).all(), label
        ref = np.asarray(_reference(s, op, a[1], b[1])).reshape(got.shape)
        total = np.asarray(_reference(s, op, np.abs(a[1]), np.abs(b[1]))).reshape(got.shape)
        tol = ((2.0 ** -22 + E) * _sum_extent(s, op) / 16 + 64 * E) * total + 5 * E * np.abs(ref) + 2.0 ** -149
        assert (np.abs(got.astype(np.float64) - ref) <= tol)[clean].all(), label


def _moved(t, offset):
    """The same operand with its block scales `offset` bytes from an aligned address, NaN bytes around them."""
    big = torch.full((t.scales.numel() + 32,), 0x7F, dtype=torch.uint8, device="cuda")
    view = big[16 + offset:16 + offset + t.scales.numel()]
    view.copy_(t.scales)
    return mq.NvfpTensor(t.codes, view, t.tensor_scale, t.fmt, t.role, t.dims)


@pytest.mark.parametrize("s", [CODES[0], CODES[1], CODES[3], CODES[4], CODES[5], MANY_TILES[1], LINEAR[2], LINEAR[13]],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fmts", [(4, 4, 4), (0, 4, 1), (2, 3, 2)])
def test_results_do_not_depend_on_the_address_of_scales(s, fmts):
    for op, (a, b) in enumerate(_operands(s, *fmts, seed=500 + sum(s))):
        a, b = a[0], b[0]
        ref = _call(s, op, a, b)
        for k, m in ((1, 0), (2, 3), (3, 1)):
            say(f"{OPS[op]} {s} {fmts}: scales at {k} and {m}")
            for fill in (0xFF, 0):
                assert torch.equal(_call(s, op, _moved(a, k), _moved(b, m), fill=fill), ref)


def test_captured_calls_with_scales_at_odd_addresses():
    s = CODES[1]
    first, second = (_operands(s, 4, 4, 4, seed) for seed in (61, 62))
    for op in range(2):
        used = [_moved(t[0], 1 + op) for t in first[op]]
        used = [mq.NvfpTensor(t.codes.clone(), t.scales, t.tensor_scale.clone(), t.fmt, t.role, t.dims) for t in used]
        ws = workspace(mq.mqconv_nvfp_gemm_workspace_bytes(s, op, 4, 4))
        refs = [_call(s, op, p[op][0][0], p[op][1][0]) for p in (first, second)]
        out = torch.empty_like(refs[0])
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream):
            FNS[op](s, *used, out, ws)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                FNS[op](s, *used, out, ws)
        for k in (1, 0, 0, 1):
            for t, new in zip(used, (first, second)[k][op]):
                for name in ("codes", "scales", "tensor_scale"):
                    getattr(t, name).copy_(getattr(new[0], name))
            out.fill_(float("nan"))
            ws.fill_(0xFF)
            torch.cuda.synchronize()
            with torch.cuda.stream(stream):
                graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, refs[k])
            FNS[op](s, *used, out, ws)


def test_injected_failures_with_scales_at_odd_addresses():
    """The launches: the scales' copy, the weights' values, the product, and, of the forward, the join of its slices."""
    s = CODES[3]
    for op, (a, b) in enumerate(_operands(s, 4, 4, 4, 63)[:2]):
        ref, moved = _call(s, op, a[0], b[0]), _moved(a[0], 3)
        try:
            launches = 4 - op
            for k in range(1, launches + 2):
                mq.mqconv_inject_launch_failure(k)
                if k <= launches:
                    with pytest.raises(mq.MqConvError) as e:
                        _call(s, op, moved, b[0])
                    assert e.value.status == -7
                else:
                    got = _call(s, op, moved, b[0])
                    mq.mqconv_inject_launch_failure(0)
                    assert torch.equal(got, ref)
        finally:
            mq.mqconv_inject_launch_failure(0)

"""include/mqconv_train.h on a machine without a GPU: exported symbols, buffer
sizes, and the refusal of every invalid argument before any HIP call; the same
tests under the host sanitizers."""
import os
import re
import subprocess
import sys

import pytest

import microscaling_quantized_convolution_mxq_amd as mq
from test_block_abi import ALIGN, FAKE, FORMAT, NULL, SHAPE, UNSUPPORTED, WORKSPACE, FakeWorkspace, _mx, _status

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mqconv_train.h")
pytestmark = pytest.mark.skipif(not os.path.exists(mq.LIB_PATH), reason="libmqconv.so not built")


def test_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(mqconv_\w+)\s*\(", src))
    out = subprocess.run(["nm", "-D", "--defined-only", mq.LIB_PATH], capture_output=True, text=True).stdout
    assert names == set(mq.EXPORTED_TRAIN)
    assert names <= set(re.findall(r"\bT\s+(mqconv_\w+)", out))


# ---- layer norm ---------------------------------------------------------------------------------
def test_layer_norm_workspace_sizes():
    for h, w, n, c in ((1, 1, 1, 1), (7, 9, 3, 45), (80, 80, 16, 64), (1, 512, 16, 4096), (1, 1, 2, 2**20), (1, 1, 2**25, 1)):
        rows = h * w * n
        ln = mq.mq_layer_norm(h, w, n, c)
        fwd, bwd = (mq.mqconv_layer_norm_workspace_bytes(ln, op) for op in (mq.NORM_FWD, mq.NORM_BWD))
        assert fwd >= 8 * rows and fwd <= 8 * rows + 16
        assert bwd >= fwd + 8 * c and bwd <= fwd + 8 * c * min(rows, 1024)
    for ln, op in ((mq.mq_layer_norm(4, 5, 3, 24), 2), (mq.mq_layer_norm(4, 5, 3, 24), -1), (mq.mq_layer_norm(0, 5, 3, 24), 0),
                   (mq.mq_layer_norm(4, 5, 3, -1), 1), (mq.mq_layer_norm(2**15, 2**15, 2, 1), 0),
                   (mq.mq_layer_norm(4, 5, 3, 24, float("nan")), 0)):
        assert mq.mqconv_layer_norm_workspace_bytes(ln, op) == 0
    with pytest.raises(mq.MqConvError):
        mq.mq_layer_norm(1, 1, 1, 2**32 + 4)


def test_layer_norm_refusals():
    ln = mq.mq_layer_norm(4, 5, 3, 24)
    ws, dims = FakeWorkspace(1 << 20), (4, 5, 3, 24)
    fwd = lambda s=ln, x=FAKE, ga=FAKE, be=FAKE, y=FAKE, m=FAKE, r=FAKE, res=None, sm=None: _status(  # noqa: E731
        mq.mqconv_layer_norm, s, x, ga, be, y, m, r, residual=res, sum=sm)
    assert fwd(x=0) == NULL and fwd(y=0) == NULL and fwd(res=FAKE) == NULL and fwd(sm=FAKE) == UNSUPPORTED
    for k in ("x", "ga", "be", "y", "m", "r"):
        assert fwd(**{k: FAKE + 2}) == ALIGN, k
    assert fwd(res=FAKE + 1, sm=FAKE) == ALIGN and fwd(res=FAKE, sm=FAKE + 2) == ALIGN
    for eps in (-1e-5, float("nan"), float("inf")):
        assert fwd(s=mq.mq_layer_norm(4, 5, 3, 24, eps)) == UNSUPPORTED
    assert fwd(s=mq.mq_layer_norm(4, 5, 0, 24)) == SHAPE and fwd(s=mq.mq_layer_norm(2**15, 2**15, 2, 1)) == SHAPE
    mx = lambda t, w=ws: _status(mq.mqconv_layer_norm_mx, ln, FAKE, FAKE, FAKE, t, ws=w)  # noqa: E731
    assert mx(_mx(mq.ROLE_GRAD, dims)) == FORMAT and mx(_mx(mq.ROLE_ACT, dims, fmt=5)) == FORMAT
    assert mx(_mx(mq.ROLE_ACT, dims, bp=16)) == UNSUPPORTED and mx(_mx(mq.ROLE_ACT, (4, 5, 3, 25))) == SHAPE
    assert mx(_mx(mq.ROLE_ACT, dims, codes=0)) == NULL and mx(_mx(mq.ROLE_ACT, dims, scales=FAKE + 8)) == ALIGN
    ok = _mx(mq.ROLE_ACT, dims)
    assert mx(ok, None) == WORKSPACE and mx(ok, FakeWorkspace(8)) == WORKSPACE and mx(ok, FakeWorkspace(1 << 20, FAKE + 8)) == ALIGN

    bwd = lambda dy=FAKE, x=FAKE, ga=FAKE, m=FAKE, r=FAKE, dx=FAKE, dg=FAKE, db=FAKE, w=ws, sk=None: _status(  # noqa: E731
        mq.mqconv_layer_norm_backward, ln, dy, x, ga, m, r, dx, dg, db, w, dskip=sk)
    for k in ("dy", "x", "m", "r", "dx"):
        assert bwd(**{k: 0}) == NULL, k
    for k in ("dy", "x", "ga", "m", "r", "dx", "dg", "db", "sk"):
        assert bwd(**{k: FAKE + 2}) == ALIGN, k
    assert bwd(w=None) == WORKSPACE and bwd(w=FakeWorkspace(64)) == WORKSPACE and bwd(w=FakeWorkspace(1 << 20, FAKE + 4)) == ALIGN
    bmx = lambda t: _status(mq.mqconv_layer_norm_backward_mx, ln, FAKE, FAKE, FAKE, FAKE, FAKE, t, ws=ws)  # noqa: E731
    assert bmx(_mx(mq.ROLE_ACT, dims)) == FORMAT and bmx(_mx(mq.ROLE_GRAD, (4, 5, 4, 24))) == SHAPE
    L = mq.train._lib()
    assert L.mqconv_layer_norm(None, FAKE, None, None, None, None, FAKE, None, None, None) == NULL
    assert L.mqconv_layer_norm_backward(None, FAKE, FAKE, None, FAKE, FAKE, None, FAKE, None, None, FAKE, 1 << 20, None) == NULL


# ---- products of two-level codes ----------------------------------------------------------------
CONV = (3, 24, 8, 9, 40, 3, 3, 2, 2, 1, 1)  # n, cin, h, w, cout, kh, kw, strides, pads: an output of 4 x 5
OPERANDS = {"x": (mq.ROLE_ACT, (8, 9, 3, 24)), "w": (mq.ROLE_WEIGHT, (40, 3, 3, 24)), "dy": (mq.ROLE_GRAD, (4, 5, 3, 40))}


def _nv(which, fmt=4, codes=FAKE, scales=FAKE, t=FAKE, role=None, dims=None):
    r, d = OPERANDS[which]
    return mq.NvfpTensor(codes, scales, t, fmt, r if role is None else role, d if dims is None else dims)


def test_product_workspace_sizes():
    ws = mq.mqconv_nvfp_gemm_workspace_bytes
    up = lambda v, m: -(-v // m) * m  # noqa: E731
    for s in (CONV, (1, 4096, 1, 1, 4096, 1, 1, 1, 1, 0, 0), (16, 64, 80, 80, 64, 3, 3, 1, 1, 1, 1), (128, 256, 20, 20, 256, 3, 3, 1, 1, 1, 1)):
        n, cin, h, w, cout, kh, kw, sh, sw, ph, pw = s
        ho, wo = (h + 2 * ph - kh) // sh + 1, (w + 2 * pw - kw) // sw + 1
        ops = (h * w * n * up(cin, 64) + cout * kh * kw * up(cin, 64), ho * wo * n * up(cout, 64) + cin * kh * kw * up(cout, 64),
               up(n, 8) * (cout * ho * wo + cin * h * w))
        outs = (ho * wo * n * cout, h * w * n * cin, cout * kh * kw * cin)
        for op in range(3):
            assert 0 < ws(s, op, 4, 4) <= 2 * ops[op] + 512 + 64 * 4 * outs[op], (s, op)
    for bad in ((CONV, 3, 4, 4), (CONV, -1, 4, 4), (CONV, 0, 5, 4), (CONV, 0, 4, -1), ((0, *CONV[1:]), 0, 4, 4),
                # 2^24 rows of 3 channels, which the products round up to 64; 2^27 pixels of one sample, rounded up to 8
                ((1, 3, 4096, 4096, 8, 1, 1, 1, 1, 0, 0), 0, 4, 4), ((1, 8, 4096, 4096, 8, 1, 1, 1, 1, 0, 0), 2, 4, 4)):
        assert ws(*bad) == 0, bad
    with pytest.raises(mq.MqConvError):
        ws((2**32 + 3, *CONV[1:]), 0, 4, 4)


def test_product_refusals():
    ws = FakeWorkspace(1 << 24)
    calls = {mq.mqconv_nvfp_forward: ("x", "w"), mq.mqconv_nvfp_backward_data: ("dy", "w"), mq.mqconv_nvfp_backward_weight: ("dy", "x")}
    for op, (fn, names) in enumerate(calls.items()):
        run = lambda a=None, b=None, out=FAKE, s=CONV, w=ws: _status(  # noqa: E731
            fn, s, a or _nv(names[0]), b or _nv(names[1]), out, w)
        for k, name in enumerate(names):
            one = lambda **kw: run(**{"ab"[k]: _nv(name, **kw)})  # noqa: E731,B023
            assert one(codes=0) == NULL and one(scales=0) == NULL and one(t=0) == NULL
            assert one(fmt=5) == FORMAT and one(fmt=-1) == FORMAT
            assert one(role=(OPERANDS[name][0] + 1) % 3) == FORMAT
            d = list(OPERANDS[name][1])
            d[3] += 1
            assert one(dims=tuple(d)) == SHAPE
            assert one(codes=FAKE + 8) == ALIGN and one(t=FAKE + 2) == ALIGN
        assert run(out=0) == NULL and run(out=FAKE + 2) == ALIGN
        assert run(w=None) == WORKSPACE and run(w=FakeWorkspace(64)) == WORKSPACE and run(w=FakeWorkspace(1 << 24, FAKE + 8)) == ALIGN
        assert run(s=(0, *CONV[1:])) == SHAPE and run(s=(*CONV[:7], 9, *CONV[8:])) == SHAPE
        L = mq.train._lib()
        a, b = (_nv(n).c_struct() for n in names)
        assert getattr(L, fn.__name__)(None, a, b, FAKE, FAKE, 1 << 24, None) == NULL
    # an operand whose rounded-up size is too large for the products
    s = (1, 3, 4096, 4096, 8, 1, 1, 1, 1, 0, 0)
    x = mq.NvfpTensor(FAKE, FAKE, FAKE, 4, mq.ROLE_ACT, (4096, 4096, 1, 3))
    w = mq.NvfpTensor(FAKE, FAKE, FAKE, 4, mq.ROLE_WEIGHT, (8, 1, 1, 3))
    assert _status(mq.mqconv_nvfp_forward, s, x, w, FAKE, ws) == SHAPE


# ---- orthogonalised update ----------------------------------------------------------------------
class FakeMatrix(FakeWorkspace):
    """An fp32 weight as the binding sees one, at an address that is never used."""

    def __init__(self, shape, at=FAKE):
        import torch
        super().__init__(4 * max(1, abs(mq._prod(shape))), at)
        self.shape, self.dtype = shape, torch.float32


def test_orthogonalize_workspace_sizes():
    ws = mq.mqconv_orthogonalize_workspace_bytes
    for shapes in ([(1, 1)], [(64, 3, 3, 64)], [(16, 27), (32, 144), (2048, 4096)], [(7, 5, 5, 3)] * 32, [(1, 10**6)], [(10**6,)]):
        up = lambda v: (v + 31) // 32 * 32  # noqa: E731
        planes = 0
        for s in shapes:
            m, n = sorted((s[0], mq._prod(s[1:])))
            planes += 4 * (3 * up(m) * up(n) + 2 * up(m) ** 2)
        assert planes < ws(shapes) <= 1.5 * planes + len(shapes) * 16384
    assert ws([]) == 0 and ws([(4, 4)] * 33) == 0 and ws([(0, 4)]) == 0 and ws([(4, -1)]) == 0
    assert ws([(23169, 23169)]) == 0 and ws([(23168, 23168)]) > 0 and ws([(32, 2**24)]) == 0 and ws([(2**30 + 1, 1)]) == 0
    with pytest.raises(mq.MqConvError):
        ws([(2**32 + 4, 4)])
    assert mq.train._lib().mqconv_orthogonalize_workspace_bytes(1, None, None) == 0


def test_update_refusals():
    ws = FakeWorkspace(1 << 20)
    M = FakeMatrix
    orth = lambda n=mq.mq_newton(), u=None, x=None, w=ws: _status(  # noqa: E731
        mq.mqconv_orthogonalize, n, [M((8, 8))] if u is None else u, [M((8, 8))] if x is None else x, w)
    assert orth(u=[], x=[]) == SHAPE and orth(u=[M((8, 8))] * 33, x=[M((8, 8))] * 33) == SHAPE
    assert orth(u=[M((8, 0))], x=[M((8, 0))]) == SHAPE and orth(x=[]) == SHAPE and orth(x=[M((4, 8))]) == SHAPE
    assert orth(u=[M((23169, 23169))], x=[M((23169, 23169))]) == SHAPE
    assert orth(u=[M((8, 8), 0)]) == NULL and orth(x=[M((8, 8), 0)]) == NULL
    assert orth(u=[M((8, 8), FAKE + 2)]) == ALIGN and orth(x=[M((8, 8), FAKE + 1)]) == ALIGN
    assert orth(w=None) == WORKSPACE and orth(w=FakeWorkspace(4096)) == WORKSPACE and orth(w=FakeWorkspace(1 << 20, FAKE + 8)) == ALIGN
    N = mq.mq_newton
    nan, inf = float("nan"), float("inf")
    for bad in (N(0), N(33), N(-1), N(5, eps=-1e-7), N(5, eps=nan), N(5, eps=inf), N(5, a=nan), N(5, b=inf), N(5, c=nan),
                # values that leave the stored range: a step's factor of 4, a polynomial that grows, one that does in its third step
                N(1, 4.0, 0.0, 0.0), N(5, 2.0, 0.0, 0.0), N(3, 1.2, 0.0, 0.0), N(1, 1.0, 3.5, 0.0), N(9, 3.9, -6.0, 3.2)):
        assert orth(n=bad) == UNSUPPORTED, (bad.steps, bad.a, bad.b, bad.c, bad.eps)
    for good in (N(), N(32), N(1, 1.5, -0.5, 0.0), N(32, 1.5, -0.5, 0.0), N(10, 15 / 8, -10 / 8, 3 / 8), N(2, 1.2, 0.0, 0.0),
                 N(12, 2.0, -1.5, 0.5), N(5, 0.0, 0.0, 0.0)):
        assert orth(n=good, w=None) == WORKSPACE, (good.steps, good.a, good.b, good.c)

    upd = lambda o=mq.mq_muon(0.1), g=None, m=None, p=None, w=ws: _status(  # noqa: E731
        mq.mqconv_muon_update, o, *([M((8, 8))] if t is None else t for t in (g, m, p)), w)
    U = mq.mq_muon
    for bad in (U(nan), U(0.1, inf), U(0.1, 0.9, nan), U(0.1, nesterov=2), U(0.1, newton=N(0))):
        assert upd(o=bad) == UNSUPPORTED
    assert upd(o=U(0.1, scale=3)) == FORMAT and upd(o=U(0.1, scale=-1)) == FORMAT and upd(o=U(0.1, rate=FAKE + 2)) == ALIGN
    for k in ("g", "m", "p"):
        assert upd(**{k: [M((8, 8), 0)]}) == NULL and upd(**{k: [M((8, 8), FAKE + 2)]}) == ALIGN
    assert upd(m=[M((8, 4))]) == SHAPE and upd(p=[]) == SHAPE and upd(w=FakeWorkspace(64)) == WORKSPACE
    L = mq.train._lib()
    assert L.mqconv_orthogonalize(None, 1, None, None, None, None, FAKE, 1 << 20, None) == NULL
    assert L.mqconv_muon_update(None, 1, None, None, None, None, None, FAKE, 1 << 20, None) == NULL
    import ctypes
    one = (ctypes.c_int32 * 1)(8)
    p = (ctypes.c_void_p * 1)(FAKE)
    assert L.mqconv_orthogonalize(ctypes.byref(N()), 1, one, one, None, p, FAKE, 1 << 20, None) == NULL
    assert L.mqconv_muon_update(ctypes.byref(U(0.1)), 1, one, one, p, None, p, FAKE, 1 << 20, None) == NULL


# ---- the same under the host sanitizers ---------------------------------------------------------
def test_refusals_under_host_sanitizers():
    if os.environ.get("MQCONV_LIB"):
        pytest.skip("already under the sanitizers")
    # (here, so that collecting the tests does not need the sanitizer build's module)
    from microscaling_quantized_convolution_mxq_amd import build_sanitize as san
    if not san.runtime():
        pytest.skip("clang AddressSanitizer runtime not installed")
    env = dict(os.environ, LD_PRELOAD=san.runtime(), MQCONV_LIB=san.build(),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert r.returncode == 0 and " passed" in out, out[-4000:]

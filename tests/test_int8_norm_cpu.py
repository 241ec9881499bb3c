"""Int8 linear and norm glue on the host: the oracle's own pins (exact rational quotients, finite
differences, brute-force sums) and every refusal of the entry points, before any HIP call."""
import ctypes
import os
from fractions import Fraction

import numpy as np
import pytest

import oracle

nf4 = pytest.importorskip("bit_nf4_quantized_codebook_amd")
lib = nf4.lib

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "nf4.h")
OK, ENULL, ESHAPE, EALIGN, EUNSUP, EWS, EHIP, EARG = 0, -1, -2, -3, -4, -5, -6, -7
FAKE = ctypes.c_void_p(0x100000)          # aligned, never dereferenced on these paths
MIS = ctypes.c_void_p(0x100004)
ODD = ctypes.c_void_p(0x100002)


# ---- the oracle against something other than itself ----

def test_int8_rows_against_rational_quotients():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 40)).astype(np.float32)
    x[1] *= 1e-30
    x[2, 5] = 300.0
    x[3] = rng.integers(-127, 128, 40) / 2          # ties: the constant becomes 0.5
    x[3, 0] = 63.5
    x[4] = 0.0
    codes, scales = oracle.int8_rows(x)
    for row in range(6):
        a = max(abs(Fraction(float(v))) for v in x[row])
        assert Fraction(float(scales[row])) == Fraction(float(np.float32(float(a) / 127.0)))
        for v, c in zip(x[row], codes[row]):
            if scales[row] == 0:
                assert c == 0
                continue
            q = Fraction(float(v)) / Fraction(float(scales[row]))
            assert max(-127, min(127, round(q))) == c          # Fraction rounds ties to even
    bad = np.ones((2, 8), np.float32)
    bad[1, 3] = np.inf
    codes, scales = oracle.int8_rows(bad)
    assert np.isnan(scales[1]) and not codes[1].any() and (codes[0] == 127).all()


def test_int8_product_brute_force():
    rng = np.random.default_rng(4)
    Xq, Wq = rng.integers(-128, 128, (3, 64)), rng.integers(-128, 128, (5, 64))
    xs, ws = rng.random(3).astype(np.float32), rng.random(5).astype(np.float32)
    got = oracle.int8_product(Xq.astype(np.int8), xs, Wq.astype(np.int8), ws)
    for m in range(3):
        for n in range(5):
            ref = sum(int(a) * int(b) for a, b in zip(Xq[m], Wq[n])) * float(xs[m]) * float(ws[n])
            assert abs(got[m, n] - ref) <= 1e-12 * abs(ref) + 1e-300


@pytest.mark.parametrize("post,gate_tokens,pre", [(True, 2, True), (False, 0, True), (True, 5, False), (False, 1, True)])
def test_norm_backward_against_differences(post, gate_tokens, pre):
    rng = np.random.default_rng(5)
    M, C = 5, 8
    draw = lambda *s: rng.standard_normal(s)  # noqa: E731
    v = {"R": draw(M, C), "B": draw(M, C)}
    if pre:
        v["w_pre"] = 1 + 0.3 * draw(C)
    if post:
        v["w_post"] = 1 + 0.3 * draw(C)
    if gate_tokens:
        v["gate"] = draw(-(-M // gate_tokens), C)
    kw = dict(gate_tokens=gate_tokens, alpha=0.75, beta=-0.5, eps=1e-3)
    dR, dH = draw(M, C), draw(M, C) if pre else None

    def loss(v):
        R, H = oracle.norm_fwd(**v, **kw)
        return (R * dR).sum() + (0 if H is None else (H * dH).sum())

    R_out, _ = oracle.norm_fwd(**v, **kw)
    par = {k: a for k, a in v.items() if k not in ("R", "B")}
    g = oracle.norm_bwd(R_out, v["B"], dR, dH, **par, **kw)
    for k, a in v.items():
        num, h = np.zeros_like(a), 1e-5
        for i in np.ndindex(a.shape):
            up, dn = ({**v, k: a + h * (np.arange(a.size).reshape(a.shape) == np.ravel_multi_index(i, a.shape)) * s}
                      for s in (1, -1))
            num[i] = (loss(up) - loss(dn)) / (2 * h)
        # central differences: h^2 times a third derivative of order 1, plus 1e-16 / h
        assert np.allclose(g["d" + k], num, rtol=0, atol=1e-7), k


def test_int8_linear_backward_is_the_linear_one_through_the_bf16_weight():
    rng = np.random.default_rng(6)
    M, N, K, r, s = 4, 8, 64, 8, 0.5
    codes, scales = oracle.int8_rows(rng.standard_normal((N, K)).astype(np.float32))
    Wb = oracle.bf16_to_f32(oracle.int8_weight_bf16(codes, scales)).astype(np.float64)
    v = {"X": rng.standard_normal((M, K)), "L1": rng.standard_normal((K, r)), "L2": rng.standard_normal((r, N))}
    dY = rng.standard_normal((M, N))
    g = oracle.backward(dY, v["X"], Wb, v["L1"], v["L2"], s)
    f = lambda v: ((v["X"] @ Wb.T + s * (v["X"] @ v["L1"]) @ v["L2"]) * dY).sum()  # noqa: E731
    for k, a in v.items():
        for i in [(0, 0), (a.shape[0] - 1, a.shape[1] - 1), (a.shape[0] // 2, 3)]:
            e = np.zeros_like(a)
            e[i] = 1e-4
            # bilinear: central differences are exact but for rounding (values of order 1e3, 1e-16 / 1e-4)
            assert abs((f({**v, k: a + e}) - f({**v, k: a - e})) / 2e-4 - g["d" + k][i]) <= 1e-8, k


# ---- refusals ----

def test_int8_quantize_refusals():
    call = lambda x=FAKE, t=0, rows=4, cols=64, codes=FAKE, scales=FAKE: lib.nf4_int8_quantize(  # noqa: E731
        x, t, rows, cols, codes, scales, None)
    assert call(t=2) == EARG and call(t=-1) == EARG
    assert call(rows=-1) == ESHAPE and call(cols=0) == ESHAPE
    assert call(cols=63) == EUNSUP and call(cols=131016) == EUNSUP and call(rows=1 << 41) == EUNSUP
    assert call(x=None, rows=0, codes=None, scales=None) == OK
    assert call(x=None) == ENULL and call(codes=None) == ENULL and call(scales=None) == ENULL
    assert call(x=MIS) == EALIGN and call(codes=MIS) == EALIGN and call(scales=ODD) == EALIGN


def _w8(rows=256, cols=256, codes=0x100000, scales=0x100000):
    return nf4._Int8Desc(codes, scales, rows, cols)


def test_limits_match_the_header():
    text = open(HEADER).read()
    assert "#define NF4_INT8_MAX_COLS 131008 " in text and "#define NF4_INT8_MAX_ROWS 2097144 " in text
    assert 131008 * 128 * 128 < 2 ** 31 <= (131008 + 64) * 128 * 128
    assert 256 * 2097144 * 4 < 2 ** 31 <= 256 * (2097144 + 8) * 4


def test_int8_weight_refusals():
    call = lambda d, out=FAKE: lib.nf4_int8_dequant(ctypes.byref(d), out, None)  # noqa: E731
    assert lib.nf4_int8_dequant(None, FAKE, None) == ENULL
    assert call(_w8(codes=None)) == ENULL and call(_w8(scales=None)) == ENULL and call(_w8(), None) == ENULL
    assert call(_w8(rows=0)) == ESHAPE and call(_w8(cols=-64)) == ESHAPE
    assert call(_w8(rows=12)) == EUNSUP and call(_w8(cols=96)) == EUNSUP and call(_w8(cols=131072)) == EUNSUP
    assert call(_w8(rows=1 << 50)) == EUNSUP
    assert call(_w8(codes=0x100008)) == EALIGN and call(_w8(scales=0x100002)) == EALIGN and call(_w8(), MIS) == EALIGN


def test_int8_linear_refusals():
    M, r = 8, 8
    wsb = lib.qlora_int8_linear_workspace_size(M, 256, 256, r)
    assert wsb > 0 and lib.qlora_int8_linear_workspace_size(0, 256, 256, r) == 0
    for bad in ((M, 256, 256, -8), (M, 256, 256, 136), (1 << 31, 256, 256, r), (M, 1 << 21, 256, r), (M, 256, 1 << 17, r)):
        assert lib.qlora_int8_linear_workspace_size(*bad) == 0

    def fwd(d=None, X=FAKE, Xq=None, xs=None, L1=FAKE, L2=FAKE, s=1.0, M=M, r=r, Y=FAKE, T=None, ws=FAKE, n=wsb):
        return lib.qlora_int8_linear_fwd(ctypes.byref(d or _w8()), X, Xq, xs, L1, L2, s, M, r, Y, T, ws, n, None)

    def bwd(d=None, dY=FAKE, X=FAKE, L1=FAKE, L2=FAKE, T=None, s=1.0, M=M, r=r, dX=FAKE, dL1=FAKE, dL2=FAKE, flags=0,
            ws=FAKE, n=wsb):
        return lib.qlora_int8_linear_bwd(ctypes.byref(d or _w8()), dY, X, L1, L2, T, s, M, r, dX, dL1, dL2, flags, ws, n,
                                         None)

    assert lib.qlora_int8_linear_fwd(None, FAKE, None, None, FAKE, FAKE, 1.0, M, r, FAKE, None, FAKE, wsb, None) == ENULL
    for f in (fwd, bwd):
        assert f(M=0) == ESHAPE and f(M=-3) == ESHAPE
        assert f(r=-8) == EUNSUP and f(r=136) == EUNSUP and f(r=12) == EUNSUP
        assert f(s=float("nan")) == EARG and f(s=float("inf")) == EARG
        assert f(_w8(cols=96)) == EUNSUP and f(_w8(rows=12)) == EUNSUP and f(_w8(rows=0)) == ESHAPE
        assert f(_w8(rows=1 << 24, cols=128)) == EUNSUP and f(M=1 << 22) == EUNSUP and f(M=1 << 40) == EUNSUP
        assert f(_w8(rows=65536), M=1 << 14) == EUNSUP
        assert f(_w8(rows=1 << 21, cols=64), M=1) == EUNSUP            # a tile row offset would pass 32 bits
        assert f(L1=None) == ENULL and f(L2=None) == ENULL and f(X=None) == ENULL
        assert f(r=0) == EARG                                   # an adapter, but no rank
        assert f(X=MIS) == EALIGN and f(L1=MIS) == EALIGN and f(L2=MIS) == EALIGN and f(ws=MIS) == EALIGN
        assert f(n=wsb - 1) == EWS and f(ws=None) == EWS
    assert fwd(Y=None) == ENULL and fwd(Y=MIS) == EALIGN and fwd(T=MIS) == EALIGN
    assert fwd(Xq=FAKE) == ENULL and fwd(xs=FAKE) == ENULL
    assert fwd(Xq=MIS, xs=FAKE) == EALIGN and fwd(Xq=FAKE, xs=ODD) == EALIGN
    assert fwd(Xq=FAKE, xs=FAKE, X=None) == ENULL              # the adapter reads X itself
    assert fwd(r=0, L1=None, L2=None, T=FAKE) == EARG
    assert fwd(r=0, L1=None, L2=None, X=None) == ENULL
    assert bwd(flags=2) == EARG and bwd(dY=None) == ENULL and bwd(dY=MIS) == EALIGN
    assert bwd(dL1=None) == ENULL and bwd(dL2=None) == ENULL and bwd(dX=MIS) == EALIGN
    none = dict(r=0, X=None, L1=None, L2=None, dL1=None, dL2=None)
    assert bwd(**none, dX=None) == ENULL and bwd(**{**none, "dL1": FAKE}) == EARG and bwd(**none, T=FAKE) == EARG


def _norm(**kw):
    d = dict(w_pre=0x100000, w_post=0x100000, gate=0x100000, gate_tokens=4, cols=256, alpha=1.0, beta=1.0, eps=1e-6,
             resid_type=0)
    d.update(kw)
    return nf4._NormDesc(*d.values())


def test_norm_refusals():
    wsb = lib.qlora_norm_workspace_size(16, 256)
    assert wsb > 0
    assert lib.qlora_norm_workspace_size(0, 256) == 0 and lib.qlora_norm_workspace_size(4, 1 << 20) == 0

    def fwd(d=None, R=FAKE, B=FAKE, M=16, Ro=FAKE, H=FAKE, Hq=None, Hs=None):
        return lib.qlora_norm_fwd(ctypes.byref(d or _norm()), R, B, M, Ro, H, Hq, Hs, None)

    def bwd(d=None, R=FAKE, B=FAKE, dRo=FAKE, dH=FAKE, M=16, dR=FAKE, dB=FAKE, dp=None, dq=None, dg=None, ws=FAKE, n=wsb):
        return lib.qlora_norm_bwd(ctypes.byref(d or _norm()), R, B, dRo, dH, M, dR, dB, dp, dq, dg, ws, n, None)

    assert lib.qlora_norm_fwd(None, FAKE, FAKE, 16, FAKE, FAKE, None, None, None) == ENULL
    for f in (fwd, bwd):
        assert f(M=0) == ESHAPE and f(M=-1) == ESHAPE and f(M=1 << 45) == EUNSUP
        assert f(_norm(cols=0)) == ESHAPE and f(_norm(cols=260)) == EUNSUP and f(_norm(cols=16392)) == EUNSUP
        assert f(_norm(resid_type=2)) == EARG
        for bad in (dict(alpha=float("nan")), dict(beta=float("inf")), dict(eps=0.0), dict(eps=-1.0),
                    dict(eps=float("nan")), dict(eps=float("inf"))):
            assert f(_norm(**bad)) == EARG, bad
        assert f(_norm(gate_tokens=0)) == ESHAPE
        assert f(_norm(w_pre=0x100004)) == EALIGN and f(_norm(w_post=0x100004)) == EALIGN
        assert f(_norm(gate=0x100004)) == EALIGN
        assert f(R=None) == ENULL and f(R=MIS) == EALIGN and f(B=MIS) == EALIGN
    pre = dict(w_post=None, gate=None)
    assert fwd(B=None) == EARG and fwd(_norm(**pre, alpha=2.0), B=None, Ro=None) == EARG
    assert fwd(_norm(**pre), B=None) == ENULL                              # R_out without B
    assert fwd(_norm(**pre, w_pre=None), B=None, Ro=None, H=None) == ENULL
    assert fwd(Ro=None) == ENULL and fwd(H=None) == ENULL and fwd(_norm(w_pre=None)) == ENULL
    assert fwd(Hq=FAKE) == ENULL and fwd(Hs=FAKE) == ENULL
    assert fwd(_norm(w_pre=None), H=None, Hq=FAKE, Hs=FAKE) == ENULL
    assert fwd(Ro=MIS) == EALIGN and fwd(H=MIS) == EALIGN and fwd(Hq=MIS, Hs=FAKE) == EALIGN
    assert fwd(Hq=FAKE, Hs=ODD) == EALIGN
    assert bwd(dH=None) == ENULL and bwd(_norm(w_pre=None)) == ENULL
    assert bwd(_norm(w_pre=None), dH=None, dRo=None) == ENULL
    assert bwd(dR=None) == ENULL and bwd(dB=None) == ENULL
    assert bwd(_norm(**pre), B=None) == ENULL                              # dB without B
    assert bwd(_norm(w_pre=None), dH=None, dp=FAKE) == EARG
    assert bwd(_norm(w_post=None), dq=FAKE) == EARG and bwd(_norm(gate=None), dg=FAKE) == EARG
    for k in ("dRo", "dH", "dR", "dB", "dp", "dq", "dg", "ws"):
        assert bwd(**{k: MIS}) == EALIGN, k
    assert bwd(n=wsb - 1) == EWS and bwd(ws=None) == EWS


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 64))
    for call in (lambda: nf4.nf4_int8_quantize(x), lambda: nf4.Int8Weight(x.to(torch.int8), x[:, 0]),
                 lambda: nf4.qlora_norm_fwd(nf4.QLoRANorm(w_pre=x[0].bfloat16()), x)):
        with pytest.raises(TypeError):
            call()

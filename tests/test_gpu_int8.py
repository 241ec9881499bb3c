"""GPU parity of the Int8 rows and the Int8 linear layer against the oracle (exact codes, float64
products), element by element.

Tolerances, from the roundings on the way (u = 2^-24, a float32 step's half; h = 2^-8, a bf16 one's):
  Y: one bf16 rounding (h |Y|); the integer sum is exact, its conversion and the two constants round
     3 u of its size; s T is rounded to bf16 (h of each of the adapter's r products) and summed in
     float32 as T is: a sum of n float32 terms is off by at most n u of the sum of their sizes.
  dX: the products are bf16 x bf16, exact in float32: (N + r + 16) u of the sizes' sum, h |dX|, and
     dT's bf16 rounding, h of the adapter's products; likewise dL2 (a sum over the tokens), and dL1,
     which takes dT in two bf16 halves, h^2.
"""
import types

import numpy as np
import pytest

import oracle
import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_nf4_quantized_codebook_amd as nf4  # noqa: E402

DEV = torch.device("cuda:0")
U, H = 2.0 ** -24, 2.0 ** -8


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def bf16(a):
    """(device bf16 tensor, its values in float64)"""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16()
    return t.to(DEV), t.double().numpy()


def f64(t):
    return t.double().cpu().numpy()


def within(name, got, ref, tol):
    got = f64(got)
    assert got.shape == ref.shape, name
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], tol[bad][:4])


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- rows to codes ----

@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 64), (5, 1000), (2, 2056), (130, 512), (7, 4096), (3, 8200), (2, 16384),
                                       (2, 28672), (1, 131008)])
def test_quantize_rows_bit_exact(rows, cols, f32):
    x = synth.normal_f32(100 + rows + cols, (rows, cols), 1.0)
    x[0, cols // 2] = -37.5
    xd = dev(x) if f32 else bf16(x)[0]
    codes, scales = nf4.nf4_int8_quantize(xd)
    rc, rs = oracle.int8_rows(f64(xd))
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), rs.view(np.uint32))


def _border_rows():
    """Rows where the code is decided next to a border: half-integer quotients (the constant a power of
    two), the floats just beside them, tiny and huge constants, denormals, zeros, signed zeros."""
    rng = np.random.default_rng(9)
    rows = []
    for scale in (0.5, 1.0, 2.0 ** -20, 2.0 ** 90, 2.0 ** -110, 2.0 ** -130):
        k = rng.integers(-126, 127, 256)
        v = (k + 0.5).astype(np.float32)
        v[::3] = np.nextafter(v[::3], np.float32(np.inf))
        v[1::3] = np.nextafter(v[1::3], np.float32(-np.inf))
        v[0] = 127.0
        rows.append((v * np.float32(scale)).astype(np.float32))
    for a in (0.7, 1.3e-20, 3.3e38, 1e-37, 2e-40, 1e-44):        # quotients beside k + 1/2 with a ragged constant
        s = np.float32(a / 127.0)
        v = ((rng.integers(-126, 127, 256) + 0.5) * float(s)).astype(np.float32)
        v[::3] = np.nextafter(v[::3], np.float32(np.inf))
        v[1::3] = np.nextafter(v[1::3], np.float32(-np.inf))
        v[0] = a
        rows.append(v)
    rows += [np.zeros(256, np.float32), np.full(256, -0.0, np.float32), np.full(256, 1e-45, np.float32),
             np.full(256, np.float32(3.4028235e38), np.float32)]
    return np.stack(rows)


def test_quantize_rows_next_to_borders():
    x = _border_rows()
    codes, scales = nf4.nf4_int8_quantize(dev(x))
    rc, rs = oracle.int8_rows(x)
    for i in range(len(x)):
        assert np.array_equal(codes[i].cpu().numpy(), rc[i]), (i, x[i][codes[i].cpu().numpy() != rc[i]])
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), rs.view(np.uint32))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_quantize_rows_not_finite(bad):
    x = synth.normal_f32(11, (4, 520), 1.0)
    x[2, 519] = bad
    for xd in (dev(x), bf16(x)[0]):
        codes, scales = nf4.nf4_int8_quantize(xd)
        clean = xd.clone()
        clean[2] = 0
        c2, s2 = nf4.nf4_int8_quantize(clean)
        assert same(codes, c2) and torch.isnan(scales[2])
        assert same(scales[[0, 1, 3]], s2[[0, 1, 3]])


def test_quantize_no_rows():
    codes, scales = nf4.nf4_int8_quantize(torch.empty((0, 64), device=DEV))
    assert codes.shape == (0, 64) and scales.shape == (0,)


@pytest.mark.parametrize("N,K", [(8, 64), (200, 320), (1032, 576)])
def test_dequant_bit_exact(N, K):
    w = nf4.Int8Weight.from_float(dev(synth.normal_f32(12, (N, K), 0.02)))
    ref = oracle.int8_weight_bf16(w.codes.cpu().numpy(), w.scales.cpu().numpy())
    assert np.array_equal(nf4.nf4_int8_dequant(w).view(torch.int16).cpu().numpy().view(np.uint16), ref)


# ---- the linear layer ----

class Lin:
    def __init__(self, seed, N, K, r):
        self.w = nf4.Int8Weight.from_float(dev(synth.heavy_tail_f32(seed, seed + 1, (N, K), 0.02, 0.2, 0.01)))
        self.Wq, self.ws = self.w.codes.cpu().numpy(), self.w.scales.cpu().numpy()
        self.L1 = self.L2 = self.l1 = self.l2 = None
        if r:
            self.L1, self.l1 = bf16(synth.normal_f32(seed + 2, (K, r), 1.0 / r))
            self.L2, self.l2 = bf16(synth.normal_f32(seed + 3, (r, N), 0.05))


def check_fwd(lin, X, s, Y, T, Xq=None):
    x = f64(X)
    codes, scales = oracle.int8_rows(x) if Xq is None else Xq
    ref = oracle.int8_product(codes, scales, lin.Wq, lin.ws)
    tol = 3 * U * np.abs(ref)
    K = x.shape[1]
    if lin.l1 is not None:
        t = x @ lin.l1
        t_tol = (K + 70) * U * (np.abs(x) @ np.abs(lin.l1))
        if T is not None:
            within("T", T, t, H * np.abs(t) + 1.01 * t_tol)
        r = lin.l1.shape[1]
        lora = np.abs(s) * (np.abs(t) @ np.abs(lin.l2))
        tol = tol + abs(s) * (t_tol @ np.abs(lin.l2)) * 1.01 + (H + (r + 8) * U) * 1.01 * lora + 2 * U * np.abs(ref)
        ref = ref + s * (t @ lin.l2)
    within("Y", Y, ref, H * (np.abs(ref) + tol) + tol)


FWD = [  # M, N, K, r
    (1, 8, 64, 0), (1, 8, 64, 8), (1, 256, 256, 16), (2, 520, 1024, 8), (3, 1032, 4096, 64), (4, 264, 8192, 128),
    (5, 4096, 320, 24), (8, 512, 1088, 64), (9, 72, 128, 8), (16, 2056, 2048, 40), (17, 264, 512, 0), (31, 1000, 704, 16),
    (33, 328, 1600, 64), (63, 600, 640, 8), (64, 512, 4096, 128), (65, 256, 256, 16), (100, 264, 192, 72),
    (128, 1040, 1024, 64), (255, 304, 576, 0), (257, 520, 320, 128), (300, 768, 2752, 64), (515, 1032, 512, 8),
    (1024, 256, 1024, 64), (1100, 520, 448, 16),
]


@pytest.mark.parametrize("M,N,K,r", FWD)
def test_linear_forward(M, N, K, r):
    print(f"int8 forward M={M} N={N} K={K} r={r}", flush=True)
    lin = Lin(2000 + M + N, N, K, r)
    X, _ = bf16(synth.heavy_tail_f32(2001 + M, 2002 + K, (M, K), 1.0, 20.0, 0.01))
    s = 16.0 / r if r else 1.0
    Y, T = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, s)
    assert (T is None) == (r == 0)
    check_fwd(lin, X, s, Y, T)
    # the codes given beforehand: the same bits
    Y2, T2 = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, s, Xq=nf4.nf4_int8_quantize(X))
    assert same(Y, Y2) and (T is None or same(T, T2))
    if not r:
        Y3, _ = nf4.qlora_int8_linear_fwd(lin.w, None, Xq=nf4.nf4_int8_quantize(X))
        assert same(Y, Y3)
    else:
        Y4, T4 = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, s, keep_T=False)
        assert T4 is None and same(Y, Y4)


@pytest.mark.parametrize("M,N,K,r", [(1, 264, 512, 8), (6, 136, 320, 0), (40, 264, 512, 16), (300, 264, 576, 8)])
def test_linear_forward_extreme_codes(M, N, K, r):
    """Every code -128 or 127 (sums at the integer range's end of this K), codes given by the caller."""
    lin = Lin(2300 + M, N, K, r)
    rng = np.random.default_rng(M)
    lin.Wq = np.where(rng.random((N, K)) < 0.9, -128, 127).astype(np.int8)
    lin.w = nf4.Int8Weight(dev(lin.Wq), lin.w.scales)
    X, _ = bf16(synth.normal_f32(2301, (M, K), 1.0))
    xq = np.where(rng.random((M, K)) < 0.9, -128, 127).astype(np.int8)
    xs = rng.random(M).astype(np.float32)
    Y, T = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5, Xq=(dev(xq), dev(xs)))
    check_fwd(lin, X, 0.5, Y, T, (xq, xs))


def test_linear_forward_longest_reduction():
    """K at its limit with every product 128 * 128: the sum is 65504 * 2^15, just inside int32."""
    for M in (1, 3, 20, 70):
        K, N = 131008, 8
        w = nf4.Int8Weight(torch.full((N, K), -128, dtype=torch.int8, device=DEV), torch.ones(N, device=DEV))
        Xq = (torch.full((M, K), -128, dtype=torch.int8, device=DEV), torch.ones(M, device=DEV))
        Y, _ = nf4.qlora_int8_linear_fwd(w, None, Xq=Xq)
        assert (Y.double() == torch.tensor(131008.0 * 16384).bfloat16().double()).all(), M


@pytest.mark.parametrize("M", [1, 5, 30, 200])
def test_linear_forward_rows_that_are_not_finite_or_zero(M):
    N, K, r = 264, 512, 8
    lin = Lin(2400, N, K, r)
    x = synth.normal_f32(2401, (M + 2, K), 1.0)
    X, _ = bf16(x)
    Y, _ = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5)
    Xb = X.clone()
    Xb[M // 2, 3] = float("nan")
    Xb[M, K - 1] = float("inf")
    Xb[M + 1] = 0
    Yb, _ = nf4.qlora_int8_linear_fwd(lin.w, Xb, lin.L1, lin.L2, 0.5)
    assert torch.isnan(Yb[M // 2]).all() and torch.isnan(Yb[M]).all() and (Yb[M + 1] == 0).all()
    keep = [m for m in range(M) if m != M // 2]
    assert same(Yb[keep], Y[keep])


# split products of every form of the sum: ranks up to 64 and beyond, few and many output groups
@pytest.mark.parametrize("M,N,K,r", [(65, 72, 4096, 8), (130, 520, 1088, 72), (90, 264, 2048, 128), (1041, 4104, 1024, 0),
                                     (1041, 4104, 1024, 24), (1041, 4104, 1024, 104)])
def test_linear_forward_split(M, N, K, r):
    print(f"int8 forward split M={M} N={N} K={K} r={r}", flush=True)
    lin = Lin(2900 + M + r, N, K, r)
    X, _ = bf16(synth.normal_f32(2901 + M, (M, K), 1.0))
    Y, T = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5)
    check_fwd(lin, X, 0.5, Y, T)


@pytest.mark.parametrize("size", [1e-30, 1e30])
@pytest.mark.parametrize("M,r", [(2, 0), (40, 16), (300, 0), (80, 64)])
def test_linear_forward_small_and_large_values(M, r, size):
    N, K = 264, 1024
    lin = Lin(2950, N, K, r)
    X, _ = bf16(np.clip(synth.normal_f32(2951, (M, K), size), -1e31, 1e31))
    Y, T = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5)
    check_fwd(lin, X, 0.5, Y, T)


def test_linear_forward_is_the_same_bits_in_any_batch():
    """Without an adapter the integer sums are exact whatever kernel or split computes them."""
    N, K = 520, 4096
    lin = Lin(2970, N, K, 0)
    X, _ = bf16(synth.normal_f32(2971, (700, K), 1.0))
    Y, _ = nf4.qlora_int8_linear_fwd(lin.w, X)
    for M in (1, 5, 17, 40, 64, 65, 200, 257, 513):
        assert same(nf4.qlora_int8_linear_fwd(lin.w, X[:M])[0], Y[:M]), M


def test_linear_forward_leaves_the_rest_alone():
    """Outputs inside larger buffers: what stands before and after them stays."""
    for M, N, K, r in ((1, 72, 128, 8), (13, 72, 128, 8), (70, 264, 192, 16), (257, 520, 128, 8)):
        lin = Lin(2500, N, K, r)
        X, _ = bf16(synth.normal_f32(2501, (M, K), 1.0))
        buf = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device=DEV)
        tb = torch.full((M + 2, r), 7.0, dtype=torch.bfloat16, device=DEV)
        Y, T = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5, Y=buf[1:M + 1], T=tb[1:M + 1])
        check_fwd(lin, X, 0.5, Y, T)
        for b in (buf, tb):
            assert (b[0] == 7).all() and (b[M + 1] == 7).all()


BWD = [(1, 8, 64, 8), (1, 264, 512, 0), (5, 520, 320, 16), (16, 264, 1088, 64), (37, 1032, 576, 128), (64, 512, 256, 8),
       (100, 264, 704, 24), (300, 776, 1024, 64), (1024, 256, 512, 16), (1100, 520, 448, 0)]


@pytest.mark.parametrize("M,N,K,r", BWD)
def test_linear_backward(M, N, K, r):
    print(f"int8 backward M={M} N={N} K={K} r={r}", flush=True)
    lin = Lin(3000 + M + N, N, K, r)
    Wb = oracle.bf16_to_f32(oracle.int8_weight_bf16(lin.Wq, lin.ws)).astype(np.float64)
    dY, dy = bf16(synth.normal_f32(3001 + M, (M, N), 1.0))
    s = 16.0 / r if r else 1.0
    size = np.abs(dy) @ np.abs(Wb)
    if not r:
        dX, dL1, dL2 = nf4.qlora_int8_linear_bwd(lin.w, dY)
        assert dL1 is None and dL2 is None
        ref = dy @ Wb
        within("dX", dX, ref, H * np.abs(ref) + 1.01 * (N + 16) * U * size)
        return
    X, x = bf16(synth.normal_f32(3002 + M, (M, K), 1.0))
    T, t = bf16(x @ lin.l1)
    dX, dL1, dL2 = nf4.qlora_int8_linear_bwd(lin.w, dY, X, lin.L1, lin.L2, T, s)
    dt = s * (dy @ lin.l2.T)
    dt_size = abs(s) * (np.abs(dy) @ np.abs(lin.l2.T))
    dt_tol = H * np.abs(dt) + 1.01 * (N + 70) * U * dt_size
    ref = dy @ Wb + dt @ lin.l1.T
    tol = 1.01 * (N + r + 16) * U * (size + np.abs(dt) @ np.abs(lin.l1.T)) + dt_tol @ np.abs(lin.l1.T)
    within("dX", dX, ref, H * (np.abs(ref) + tol) + tol)
    ref = x.T @ dt
    # dL1 takes dT as two bf16 values: H of a rest that is at most H of it
    rest = H * H * np.abs(dt) + 1.01 * (N + 70) * U * dt_size
    tol = 1.01 * (2 * M + 70) * U * (np.abs(x).T @ np.abs(dt)) + np.abs(x).T @ rest
    within("dL1", dL1, ref, H * (np.abs(ref) + tol) + tol)
    ref = s * (t.T @ dy)
    tol = 1.01 * (M + 70) * U * abs(s) * (np.abs(t).T @ np.abs(dy))
    within("dL2", dL2, ref, H * (np.abs(ref) + tol) + tol)
    # T left out: computed again, to bf16 of the same sums (their order may differ by a rounding)
    again = nf4.qlora_int8_linear_bwd(lin.w, dY, X, lin.L1, lin.L2, None, s)
    assert same(again[0], dX) and same(again[1], dL1)
    t_tol = 2 * H * np.abs(t) + 1.01 * (K + 70) * U * (np.abs(x) @ np.abs(lin.l1))
    tol = tol + abs(s) * (t_tol.T @ np.abs(dy))
    within("dL2 (T again)", again[2], ref, H * (np.abs(ref) + tol) + tol)
    # without dX; and added to what is there (the sum in float32, one rounding)
    none, dL1b, dL2b = nf4.qlora_int8_linear_bwd(lin.w, dY, X, lin.L1, lin.L2, T, s, need_dX=False)
    assert none is None and same(dL1b, dL1) and same(dL2b, dL2)
    base, bv = bf16(synth.normal_f32(3003, (M, K), 3.0))
    acc, _, _ = nf4.qlora_int8_linear_bwd(lin.w, dY, X, lin.L1, lin.L2, T, s, dX=base, accumulate=True)
    ref = dy @ Wb + dt @ lin.l1.T + bv
    tol = 1.01 * (N + r + 17) * U * (size + np.abs(dt) @ np.abs(lin.l1.T) + np.abs(bv)) + dt_tol @ np.abs(lin.l1.T)
    within("dX accumulated", acc, ref, H * (np.abs(ref) + tol) + tol)


@pytest.mark.parametrize("M", [3, 300, 4096])
def test_linear_backward_with_the_largest_constants(M):
    """Constants next to FLT_MAX / 127: a weight's value fits bf16, 128 constants do not fit float32."""
    N, K = 512, 512
    codes = np.random.default_rng(31).integers(-127, 128, (N, K)).astype(np.int8)
    scales = np.linspace(2.6e36, 2.66e36, N).astype(np.float32)
    w = nf4.Int8Weight(dev(codes), dev(scales))
    Wb = oracle.bf16_to_f32(oracle.int8_weight_bf16(codes, scales)).astype(np.float64)
    assert np.isfinite(Wb).all()
    dY, dy = bf16(synth.normal_f32(3100 + M, (M, N), 1e-10))
    dX, _, _ = nf4.qlora_int8_linear_bwd(w, dY)
    ref = dy @ Wb
    tol = 1.01 * (N + 16) * U * (np.abs(dy) @ np.abs(Wb))
    within("dX", dX, ref, H * (np.abs(ref) + tol) + tol)


def test_linear_repeats_bit_for_bit_and_with_a_dirty_workspace():
    for M, N, K, r in ((1, 1032, 4096, 64), (20, 520, 2048, 16), (200, 520, 4096, 64), (1100, 520, 1024, 8)):
        lin = Lin(4000, N, K, r)
        X, _ = bf16(synth.normal_f32(4001, (M, K), 1.0))
        dY, _ = bf16(synth.normal_f32(4002, (M, N), 1.0))
        n = nf4.qlora_int8_linear_workspace_size(M, N, K, r)
        first = None
        for fill in (0, 0x7F, 0xFF):
            ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
            Y, T = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5, workspace=ws)
            ws.fill_(fill)
            out = (Y, T) + nf4.qlora_int8_linear_bwd(lin.w, dY, X, lin.L1, lin.L2, T, 0.5, workspace=ws)
            first = first or out
            assert all(same(a, b) for a, b in zip(first, out)), (M, fill)


def test_linear_on_a_side_stream_and_two_at_once():
    M, N, K, r = 12, 520, 2048, 16
    lin = Lin(4100, N, K, r)
    X, _ = bf16(synth.normal_f32(4101, (M, K), 1.0))
    ref, _ = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    torch.cuda.synchronize()
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5)[0])
    torch.cuda.synchronize()
    assert all(same(ref, y) for y in got)


@pytest.mark.parametrize("M", [1, 16, 300, 1100])
def test_linear_step_captured_and_replayed(M):
    N, K, r = 520, 1024, 16
    lin = Lin(4200, N, K, r)
    X, _ = bf16(synth.normal_f32(4201, (M, K), 1.0))
    dY, _ = bf16(synth.normal_f32(4202, (M, N), 1.0))

    def step():
        Y, T = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5)
        return (Y, T) + nf4.qlora_int8_linear_bwd(lin.w, dY, X, lin.L1, lin.L2, T, 0.5)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for rep in range(3):
        X.copy_(bf16(synth.normal_f32(4210 + rep, (M, K), 1.0))[0])
        dY.copy_(bf16(synth.normal_f32(4220 + rep, (M, N), 1.0))[0])
        g.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, step())), rep
        torch.cuda.synchronize()


@pytest.mark.parametrize("rows,cols", [((1 << 21) + 5, 64), (1_100_003, 4096)])
def test_quantize_more_rows_than_a_launch_takes_and_offsets_past_32_bits(rows, cols):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(rows)
    X = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV).normal_(0, 1, generator=gen)
    codes, scales = nf4.nf4_int8_quantize(X)
    for part in (slice(0, 3), slice((1 << 20) - 2, (1 << 20) + 2), slice(rows - 5, rows)):
        rc, rs = oracle.int8_rows(f64(X[part]))
        assert np.array_equal(codes[part].cpu().numpy(), rc) and np.array_equal(scales[part].cpu().numpy(), rs)


def test_linear_with_operands_just_below_2_gib():
    """X of 2^31 - 8192 bytes; a weight of more rows than 2^20: the last rows and columns against the oracle."""
    M, N, K, r = 262143, 64, 4096, 8
    lin = Lin(4400, N, K, r)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    X = torch.empty((M, K), dtype=torch.bfloat16, device=DEV).normal_(0, 1, generator=gen)
    Y, T = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5)
    dX, dL1, dL2 = nf4.qlora_int8_linear_bwd(lin.w, Y, X, lin.L1, lin.L2, T, 0.5)
    Wb = oracle.bf16_to_f32(oracle.int8_weight_bf16(lin.Wq, lin.ws)).astype(np.float64)
    for part in (slice(0, 3), slice(M - 3, M)):
        check_fwd(lin, X[part], 0.5, Y[part], T[part])
        dy = f64(Y[part])
        dt = 0.5 * (dy @ lin.l2.T)
        ref = dy @ Wb + dt @ lin.l1.T
        size = np.abs(dy) @ np.abs(Wb) + np.abs(dt) @ np.abs(lin.l1.T)
        dt_tol = H * np.abs(dt) + 1.01 * (N + 70) * U * 0.5 * (np.abs(dy) @ np.abs(lin.l2.T))
        tol = 1.01 * (N + r + 16) * U * size + dt_tol @ np.abs(lin.l1.T)
        within("dX", dX[part], ref, H * (np.abs(ref) + tol) + tol)
    del X, dX, Y, T
    N, K = (1 << 20) + 8, 64
    w = nf4.Int8Weight.from_float(torch.empty((N, K), device=DEV).normal_(0, 1, generator=gen))
    for M in (1, 3, 20, 65):
        X, x = bf16(synth.normal_f32(4401 + M, (M, K), 1.0))
        Y, _ = nf4.qlora_int8_linear_fwd(w, X)
        part = slice(N - 40, N)
        ref = oracle.int8_product(*oracle.int8_rows(x), w.codes[part].cpu().numpy(), w.scales[part].cpu().numpy())
        within("Y", Y[:, part], ref, H * np.abs(ref) * 1.01 + 3 * U * np.abs(ref))
        dX, _, _ = nf4.qlora_int8_linear_bwd(w, Y)
        # a sum of 2^20 terms: against float64 on the device (a product of two contiguous float64 matrices)
        Wd = (w.codes.float() * w.scales[:, None]).bfloat16().double()
        ref, size = torch.mm(Y.double(), Wd), torch.mm(Y.double().abs(), Wd.abs())
        within("dX", dX, f64(ref), H * np.abs(f64(ref)) * 1.01 + 1.01 * (N + 16) * U * f64(size))


def test_weight_tensors_cannot_be_replaced():
    w = nf4.Int8Weight(torch.zeros((8, 64), dtype=torch.int8, device=DEV), torch.zeros(8, device=DEV))
    with pytest.raises(AttributeError):
        w.codes = w.codes[:4]


def test_binding_refusals():
    lin = Lin(4300, 64, 128, 8)
    X, _ = bf16(np.ones((4, 128)))
    for bad in (lambda: nf4.qlora_int8_linear_fwd(lin.w, X.t().contiguous(), lin.L1, lin.L2),
                lambda: nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2[:, :56].contiguous()),
                lambda: nf4.qlora_int8_linear_fwd(lin.w, X[:, ::2]),
                lambda: nf4.qlora_int8_linear_fwd(lin.w, X, T=X),
                lambda: nf4.qlora_int8_linear_fwd(lin.w, X, Y=X),
                lambda: nf4.qlora_int8_linear_bwd(lin.w, X[:, :64].contiguous(), accumulate=True),
                lambda: nf4.qlora_int8_linear_fwd(lin.w, X, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)),
                lambda: nf4.qlora_int8_linear_fwd(lin.w, X, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
                lambda: nf4.Int8Weight(lin.w.codes, lin.w.scales[:8])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nf4.qlora_int8_linear_fwd(lin.w, X.float()), lambda: nf4.nf4_int8_quantize(X.half()),
                lambda: nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, None), lambda: nf4.Int8Weight(lin.w.codes.int(), None)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(nf4.NF4Error):
        nf4.qlora_int8_linear_fwd(lin.w, X[:0])
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_int8_quantize(torch.zeros((2, 12), device=DEV))


def test_binding_refuses_a_missing_x():
    lin = Lin(4400, 64, 128, 8)
    X, _ = bf16(np.ones((4, 128)))
    Xq = nf4.nf4_int8_quantize(X)
    for bad in (lambda: nf4.qlora_int8_linear_fwd(lin.w, None), lambda: nf4.qlora_int8_linear_fwd(lin.w, None, lin.L1, lin.L2, Xq=Xq)):
        with pytest.raises(ValueError):
            bad()
    assert same(nf4.qlora_int8_linear_fwd(lin.w, None, Xq=Xq)[0], nf4.qlora_int8_linear_fwd(lin.w, X)[0])


# every form of the forward: GEMV with 1, 2 and 4 groups of tokens, loads of its own and through LDS, 4 and 8
# waves; the product whole, with one and two adapter steps; the split product's sum
ADAPTER = [(1, 264, 512, 8), (3, 520, 1024, 128), (12, 520, 320, 64), (16, 264, 2048, 16), (29, 264, 512, 40),
           (40, 264, 576, 128), (64, 520, 1024, 72), (3, 8200, 320, 8), (9, 8200, 320, 24), (20, 8200, 320, 16),
           (40, 8200, 320, 72), (50, 16392, 192, 8), (100, 264, 192, 64), (257, 520, 320, 16), (100, 264, 192, 72),
           (600, 520, 320, 128), (65, 72, 4096, 8), (130, 520, 1088, 72), (1041, 4104, 1024, 24)]


@pytest.mark.parametrize("M,N,K,r", ADAPTER)
def test_linear_forward_adapter_alone(M, N, K, r):
    """A weight of zeros: Y is the adapter's term, rounded once.  s T enters it as two bf16 halves: the second
    is off by at most h of a rest that is at most h of s T, so the term by h^2 of its products' sizes; its 2 r
    products are summed in float32, and T as in check_fwd."""
    print(f"int8 forward, adapter alone M={M} N={N} K={K} r={r}", flush=True)
    w = nf4.Int8Weight(torch.zeros((N, K), dtype=torch.int8, device=DEV), torch.ones(N, device=DEV))
    L1, l1 = bf16(synth.normal_f32(5000 + K, (K, r), 1.0 / r))
    L2, l2 = bf16(synth.normal_f32(5001 + N, (r, N), 0.05))
    X, x = bf16(synth.normal_f32(5002 + M, (M, K), 1.0))
    s = 0.75
    Y, T = nf4.qlora_int8_linear_fwd(w, X, L1, L2, s)
    t = x @ l1
    t_tol = 1.01 * (K + 70) * U * (np.abs(x) @ np.abs(l1))
    within("T", T, t, H * (np.abs(t) + t_tol) + t_tol)
    ref = s * (t @ l2)
    tol = s * (t_tol @ np.abs(l2)) + 1.01 * (H * H + (2 * r + 16) * U) * s * (np.abs(t) @ np.abs(l2))
    within("Y", Y, ref, H * (np.abs(ref) + tol) + tol)


def plan(M, N, K):
    """The backward's route for this shape: whether dX's product expands the weight to bf16 first or converts
    its codes on the way, and over how many workgroups its reduction is split.  Both follow from the workspace
    size, which holds the expansion and the splits' partials: of the two routes exactly one has that size."""
    def split(tiles, steps):
        s = max(1, min(256 // tiles, steps // 4, 16))
        per = -(-steps // s)
        per = -(-per // 4) * 4
        return max(1, -(-steps // per))

    up = lambda n: -(-n // 256) * 256  # noqa: E731
    tiles = lambda rows, cols: -(-M // rows) * -(-cols // 256)  # noqa: E731
    fwd = 1 if M <= 64 else split(tiles(256, N), -(-K // 128))
    steps = -(-N // 64)
    got = {}
    for route, s in (("expand", split(tiles(256, K), steps)), ("convert", split(tiles(64 if M <= 64 else 128, K), steps))):
        partials = max(s * M * K if s > 1 else 0, fwd * M * N if fwd > 1 else 0)
        got[up(M * K) + up(4 * M) + (up(2 * N * K) if route == "expand" else 0) + up(4 * partials)] = (route, s)
    assert len(got) == 2, "the size does not tell the routes apart"
    return got[nf4.qlora_int8_linear_workspace_size(M, N, K, 0)]


@pytest.mark.parametrize("M,N,K,r,route,split", [
    (37, 1032, 576, 128, "convert", 3), (20, 520, 2048, 16, "convert", 2), (200, 520, 4096, 64, "convert", 2),
    (37, 264, 1472, 72, "convert", 1), (300, 200, 3136, 8, "convert", 1), (16, 264, 1088, 64, "expand", 1),
    (100, 1032, 320, 24, "expand", 3), (300, 520, 320, 128, "expand", 2), (1100, 264, 448, 72, "expand", 1)])
def test_linear_backward_adapter_alone(M, N, K, r, route, split):
    """A weight of zeros: dX is the adapter's term, rounded once.  dT enters it as two bf16 halves (h^2 of its
    products' sizes); its 2 r products are summed in float32, dT's as in test_linear_backward."""
    print(f"int8 backward, adapter alone M={M} N={N} K={K} r={r}", flush=True)
    assert plan(M, N, K) == (route, split)
    w = nf4.Int8Weight(torch.zeros((N, K), dtype=torch.int8, device=DEV), torch.ones(N, device=DEV))
    L1, l1 = bf16(synth.normal_f32(5100 + K, (K, r), 1.0 / r))
    L2, l2 = bf16(synth.normal_f32(5101 + N, (r, N), 0.05))
    X, x = bf16(synth.normal_f32(5102 + M, (M, K), 1.0))
    dY, dy = bf16(synth.normal_f32(5103 + M, (M, N), 1.0))
    T, _ = bf16(x @ l1)
    s = 0.75
    dX, _, _ = nf4.qlora_int8_linear_bwd(w, dY, X, L1, L2, T, s)
    dt = s * (dy @ l2.T)
    dt_tol = 1.01 * (N + 70) * U * s * (np.abs(dy) @ np.abs(l2.T))
    ref = dt @ l1.T
    tol = dt_tol @ np.abs(l1.T) + 1.01 * (H * H + (2 * r + 16) * U) * (np.abs(dt) @ np.abs(l1.T))
    within("dX", dX, ref, H * (np.abs(ref) + tol) + tol)
    base, bv = bf16(synth.normal_f32(5104, (M, K), 0.25))
    acc, _, _ = nf4.qlora_int8_linear_bwd(w, dY, X, L1, L2, T, s, dX=base, accumulate=True)
    ref, tol = ref + bv, tol + 2 * U * np.abs(bv)
    within("dX accumulated", acc, ref, H * (np.abs(ref) + tol) + tol)


@pytest.mark.parametrize("int8", [True, False])
def test_linear_backward_with_more_than_2_gib_of_T(int8):
    """T's limit is not X's: 128 columns against X's 64, so T passes 2 GiB while X and dY stay below.  All rows
    are zero but the first and the last ones, so that the sums over the tokens have 27 terms."""
    M, N, K, r, s = (1 << 23) + 24, 64, 64, 128, 0.5
    W = dev(synth.normal_f32(5200, (N, K), 0.05))
    w = nf4.Int8Weight.from_float(W) if int8 else nf4.NF4Weight.from_float(W)
    L1, l1 = bf16(synth.normal_f32(5201, (K, r), 0.1))
    L2, l2 = bf16(synth.normal_f32(5202, (r, N), 0.1))
    live = torch.cat([torch.arange(3), torch.arange(M - 24, M)]).to(DEV)

    def rows(seed, cols):
        full = torch.zeros((M, cols), dtype=torch.bfloat16, device=DEV)
        full[live], v = bf16(synth.normal_f32(seed, (27, cols), 1.0))
        return full, v

    X, x = rows(5203, K)
    dY, dy = rows(5204, N)
    T, t = rows(5205, r)
    if int8:
        lin = types.SimpleNamespace(l1=l1, l2=l2, Wq=w.codes.cpu().numpy(), ws=w.scales.cpu().numpy())
        Y, T_out = nf4.qlora_int8_linear_fwd(w, X, L1, L2, s)
        check_fwd(lin, X[live], s, Y[live], T_out[live])
        del Y, T_out
    bwd = nf4.qlora_int8_linear_bwd if int8 else nf4.qlora_linear_bwd
    _, dL1, dL2 = bwd(w, dY, X, L1, L2, T, s, need_dX=False)
    dt = s * (dy @ l2.T)
    # dT's own rounding: two bf16 halves (h^2) in the Int8 layer, one (h) in the other
    rest = (H * H if int8 else H) * np.abs(dt) + 1.01 * (N + 70) * U * s * (np.abs(dy) @ np.abs(l2.T))
    ref = x.T @ dt
    tol = np.abs(x).T @ rest + 1.01 * (2 * 27 + 70) * U * (np.abs(x).T @ np.abs(dt))
    within("dL1", dL1, ref, H * (np.abs(ref) + tol) + tol)
    ref = s * (t.T @ dy)
    tol = 1.01 * (27 + 70) * U * s * (np.abs(t).T @ np.abs(dy))
    within("dL2", dL2, ref, H * (np.abs(ref) + tol) + tol)


@pytest.mark.parametrize("M,N,K,route,split", [
    (37, 1032, 576, "convert", 3), (200, 520, 4096, "convert", 2), (37, 264, 1472, "convert", 1),
    (300, 200, 3136, "convert", 1), (300, 520, 320, "expand", 2), (1100, 264, 448, "expand", 1)])
def test_linear_backward_with_the_largest_constants_on_every_route(M, N, K, route, split):
    """Constants next to FLT_MAX / 127 through both products and their splits: 128 constants, or a code turned
    to an unsigned byte times its constant, do not fit float32; the weight's values do."""
    assert plan(M, N, K) == (route, split)
    codes = np.random.default_rng(32).integers(-127, 128, (N, K)).astype(np.int8)
    scales = np.linspace(2.6e36, 2.66e36, N).astype(np.float32)
    w = nf4.Int8Weight(dev(codes), dev(scales))
    Wb = oracle.bf16_to_f32(oracle.int8_weight_bf16(codes, scales)).astype(np.float64)
    assert np.isfinite(Wb).all()
    dY, dy = bf16(synth.normal_f32(5300 + M, (M, N), 1e-10))
    dX, _, _ = nf4.qlora_int8_linear_bwd(w, dY)
    ref = dy @ Wb
    tol = 1.01 * (N + 16) * U * (np.abs(dy) @ np.abs(Wb))
    within("dX", dX, ref, H * (np.abs(ref) + tol) + tol)


def guarded(shape, guard, value=7.0):
    """(buffer, view): the view lies between `guard` rows of one value on each side."""
    buf = torch.full((shape[0] + 2 * guard, shape[1]), value, dtype=torch.bfloat16, device=DEV)
    return buf, buf[guard:guard + shape[0]]


def untouched(buf, guard, value=7.0):
    return bool((buf[:guard] == value).all()) and bool((buf[-guard:] == value).all())


# Both converting tiles with the reduction unsplit (stores to dX itself) and split, and the expanded product; M
# ragged against the tile's rows, K against its 256 columns, ranks of none, one and two adapter steps.
@pytest.mark.parametrize("M,N,K,r,route,split", [
    (37, 264, 1472, 0, "convert", 1), (37, 264, 2112, 72, "convert", 1), (64, 264, 1472, 8, "convert", 1),
    (130, 328, 1984, 0, "convert", 1), (300, 200, 3136, 128, "convert", 1), (600, 392, 1600, 24, "convert", 1),
    (37, 1032, 576, 16, "convert", 3), (200, 520, 4096, 72, "convert", 2), (300, 520, 320, 16, "expand", 2),
    (1100, 264, 448, 72, "expand", 1), (1100, 520, 448, 0, "expand", 2)])
def test_linear_backward_writes_its_outputs_and_nothing_else(M, N, K, r, route, split):
    """dX, dL1 and dL2 inside larger buffers, with 256 rows (a tile's) of a value on each side; dX written, then
    added to.  Tolerances as in test_linear_backward, with dT in two halves."""
    print(f"int8 backward in guarded buffers M={M} N={N} K={K} r={r}", flush=True)
    assert plan(M, N, K) == (route, split)
    lin = Lin(5400 + M + N, N, K, r)
    Wb = oracle.bf16_to_f32(oracle.int8_weight_bf16(lin.Wq, lin.ws)).astype(np.float64)
    dY, dy = bf16(synth.normal_f32(5401 + M, (M, N), 1.0))
    bX, dX = guarded((M, K), 256)
    start = synth.normal_f32(5402 + M, (M, K), 2.0)
    ref, size, inner, s = dy @ Wb, np.abs(dy) @ np.abs(Wb), 0.0, 0.5
    args, kw = (), {}
    if r:
        X, x = bf16(synth.normal_f32(5403 + M, (M, K), 1.0))
        T, t = bf16(x @ lin.l1)
        b1, dL1 = guarded((K, r), 256)
        b2, dL2 = guarded((r, N), 256)
        args, kw = (X, lin.L1, lin.L2, T, s), dict(dL1=dL1, dL2=dL2)
        dt = s * (dy @ lin.l2.T)
        rest = H * H * np.abs(dt) + 1.01 * (N + 70) * U * s * (np.abs(dy) @ np.abs(lin.l2.T))
        ref, size, inner = ref + dt @ lin.l1.T, size + np.abs(dt) @ np.abs(lin.l1.T), rest @ np.abs(lin.l1.T)
    for accumulate in (False, True):
        base = np.zeros((M, K))
        if accumulate:
            v, base = bf16(start)
            dX.copy_(v)
        got = nf4.qlora_int8_linear_bwd(lin.w, dY, *args, dX=dX, accumulate=accumulate, **kw)
        assert got[0] is dX
        tol = 1.01 * (N + 2 * r + 17) * U * (size + np.abs(base)) + inner
        within("dX", dX, ref + base, H * (np.abs(ref + base) + tol) + tol)
        assert untouched(bX, 256)
        if r:
            want = x.T @ dt
            tol = np.abs(x).T @ rest + 1.01 * (2 * M + 70) * U * (np.abs(x).T @ np.abs(dt))
            within("dL1", dL1, want, H * (np.abs(want) + tol) + tol)
            want = s * (t.T @ dy)
            tol = 1.01 * (M + 70) * U * s * (np.abs(t).T @ np.abs(dy))
            within("dL2", dL2, want, H * (np.abs(want) + tol) + tol)
            assert untouched(b1, 256) and untouched(b2, 256)


# The GEMV's forms of wide weights (from 8192 rows: 4 waves, or 8 with 32 rows; from 16384: 4 waves with 32
# rows), with an adapter; and T's partials past 64 MiB in all workgroups together, where T is summed by a
# launch of its own.
@pytest.mark.parametrize("M,N,K,r", [(3, 8200, 320, 8), (3, 8200, 64, 128), (9, 8200, 320, 24), (16, 16392, 128, 40),
                                     (20, 8200, 320, 16), (32, 16392, 192, 128), (40, 8200, 320, 72), (64, 8200, 576, 8),
                                     (50, 16392, 192, 8), (64, 16392, 64, 64), (64, 8200, 2048, 128), (16, 28680, 2112, 128)])
def test_linear_forward_few_tokens_wide_weights(M, N, K, r):
    print(f"int8 forward, wide M={M} N={N} K={K} r={r}", flush=True)
    lin = Lin(5500 + M + K, N, K, r)
    X, _ = bf16(synth.heavy_tail_f32(5501 + M, 5502 + K, (M, K), 1.0, 20.0, 0.01))
    by, Y = guarded((M, N), 64)
    bt, T = guarded((M, r), 64)
    nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5, Y=Y, T=T)
    check_fwd(lin, X, 0.5, Y, T)
    assert untouched(by, 64) and untouched(bt, 64)
    # the same rows through all of it again, without T
    Y2, none = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5, keep_T=False)
    assert none is None and same(Y2, Y)


@pytest.mark.parametrize("M,N,K,r", [(1, 72, 128, 8), (5, 264, 512, 0), (13, 72, 128, 8), (33, 264, 576, 72), (70, 264, 192, 16),
                                     (129, 520, 128, 72), (257, 520, 128, 8), (300, 776, 320, 0), (65, 72, 4096, 8),
                                     (257, 264, 2048, 128), (1041, 4104, 1024, 24)])
def test_linear_forward_leaves_a_tile_around_its_outputs_alone(M, N, K, r):
    """256 rows on each side, as many as a tile of the product has: rows of a tile past M are not written."""
    lin = Lin(5600 + M, N, K, r)
    X, _ = bf16(synth.normal_f32(5601 + M, (M, K), 1.0))
    by, Y = guarded((M, N), 256)
    bt, T = guarded((M, r), 256) if r else (None, None)
    nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5, Y=Y, T=T)
    check_fwd(lin, X, 0.5, Y, T)
    assert untouched(by, 256) and (not r or untouched(bt, 256))


@pytest.mark.parametrize("M,N,K,r", [(3, 72, 128, 8), (40, 264, 576, 128), (65, 72, 4096, 8), (200, 520, 4096, 72), (257, 520, 320, 16),
                                     (300, 520, 320, 128), (1100, 264, 448, 72)])
def test_linear_stays_inside_its_workspace(M, N, K, r):
    lin = Lin(5700 + M, N, K, r)
    X, _ = bf16(synth.normal_f32(5701 + M, (M, K), 1.0))
    dY, _ = bf16(synth.normal_f32(5702 + M, (M, N), 1.0))
    n, guard = nf4.qlora_int8_linear_workspace_size(M, N, K, r), 4 << 20
    buf = torch.full((n + 2 * guard,), 0x5A, dtype=torch.uint8, device=DEV)
    ws = buf[guard:guard + n]
    Y, T = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5, workspace=ws)
    nf4.qlora_int8_linear_bwd(lin.w, dY, X, lin.L1, lin.L2, T, 0.5, workspace=ws)
    nf4.qlora_int8_linear_bwd(lin.w, dY, X, lin.L1, lin.L2, None, 0.5, workspace=ws)
    check_fwd(lin, X, 0.5, Y, T)
    assert (buf[:guard] == 0x5A).all() and (buf[guard + n:] == 0x5A).all()


@pytest.mark.parametrize("M,N,K,r,route", [(37, 264, 1472, 72, "convert"), (200, 520, 4096, 16, "convert"), (300, 520, 320, 8, "expand"),
                                           (1100, 264, 448, 0, "expand")])
def test_linear_backward_rows_that_are_not_finite(M, N, K, r, route):
    """A token with a NaN or an infinity in dY, or in X, leaves the other tokens' dX as they are."""
    assert plan(M, N, K)[0] == route
    lin = Lin(5800 + M, N, K, r)
    dY, _ = bf16(synth.normal_f32(5801, (M, N), 1.0))
    X, x = bf16(synth.normal_f32(5802, (M, K), 1.0))
    args = (X, lin.L1, lin.L2, bf16(x @ lin.l1)[0], 0.5) if r else ()
    clean = nf4.qlora_int8_linear_bwd(lin.w, dY, *args)[0]
    dY[3, 5] = float("nan")
    dY[M - 1, N - 1] = float("-inf")
    if r:
        X[4, 7] = float("inf")
    got = nf4.qlora_int8_linear_bwd(lin.w, dY, *args)[0]
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[M - 1]).any()
    keep = [m for m in range(M) if m not in (3, M - 1)]
    assert same(got[keep], clean[keep])


def test_linear_forward_channels_that_are_not_finite():
    """A weight row with constant NaN (nf4_int8_quantize's for a row that is not finite), or an infinity in a
    column of L2, concerns its own output channel."""
    N, K, r = 264, 512, 8
    lin = Lin(5900, N, K, r)
    scales, L2 = lin.w.scales.clone(), lin.L2.clone()
    scales[17] = float("nan")
    L2[3, 100] = float("inf")
    bad = nf4.Int8Weight(lin.w.codes, scales)
    for M in (1, 7, 20, 40, 70, 300):
        X, _ = bf16(synth.normal_f32(5901 + M, (M, K), 1.0))
        Y, _ = nf4.qlora_int8_linear_fwd(lin.w, X, lin.L1, lin.L2, 0.5)
        got, _ = nf4.qlora_int8_linear_fwd(bad, X, lin.L1, L2, 0.5)
        assert torch.isnan(got[:, 17]).all() and not torch.isfinite(got[:, 100]).any(), M
        keep = [n for n in range(N) if n not in (17, 100)]
        assert same(got[:, keep], Y[:, keep]), M

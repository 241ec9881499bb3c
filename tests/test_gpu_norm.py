"""GPU parity of the norm glue between blocks against the float64 oracle, element by element, and a
decoder block's run of it with the Int8 linears.

Tolerances, from the roundings on the way (u = 2^-24, h = 2^-8): a row's sum of C squares is off by
at most (C/NT + 32) u of itself (positive terms; NT threads add a few each, then trees), so 1/rms by
half of that and a few u: E = 64 u covers every size here (at most 32 elements a thread).  Each
output adds its type's rounding (h for bf16, 2 u for float32) and E of the sizes of its terms; the
sums over tokens add (M + 32) u of the sizes' sum.
"""
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
E = 64 * U


def f64(t):
    return t.double().cpu().numpy()


def within(name, got, ref, tol):
    got = f64(got)
    assert got.shape == ref.shape, name
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4], tol[bad][:4])


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


class Case:
    def __init__(self, M, C, pre=True, post=True, gate=0, f32=False, block=True, seed=0, alpha=0.875, beta=-0.375):
        n = lambda k, shape, std: torch.from_numpy(synth.normal_f32(7000 + 50 * seed + k, shape, std)).to(DEV)  # noqa: E731
        self.res = torch.float32 if f32 else torch.bfloat16
        self.R = n(0, (M, C), 2.0).to(self.res)
        self.B = n(1, (M, C), 0.7).bfloat16() if block else None
        v = lambda k: (1 + n(k, (C,), 0.2)).bfloat16()  # noqa: E731
        self.norm = nf4.QLoRANorm(w_pre=v(2) if pre else None, w_post=v(3) if post else None, eps=1e-5)
        if block:
            self.norm.alpha, self.norm.beta = alpha, beta
        if gate:
            self.norm.gate, self.norm.gate_tokens = n(4, (-(-M // gate), C), 0.5).bfloat16(), gate
        self.dR = n(5, (M, C), 1.0).to(self.res)
        self.dH = n(6, (M, C), 1.0).bfloat16() if pre else None

    def params(self):
        p = self.norm
        a = lambda t: None if t is None else f64(t)  # noqa: E731
        return dict(w_pre=a(p.w_pre), w_post=a(p.w_post), gate=a(p.gate), gate_tokens=p.gate_tokens, alpha=float(p.alpha),
                    beta=float(p.beta), eps=float(np.float32(p.eps)))

    def check_fwd(self):
        kw = self.params()
        R, B = f64(self.R), None if self.B is None else f64(self.B)
        ref_R, ref_H = oracle.norm_fwd(R, B, **kw)
        Ro, Hh = nf4.qlora_norm_fwd(self.norm, self.R, self.B)
        size = np.abs(R)
        if B is None:
            assert Ro is None
        else:
            size = abs(kw["alpha"]) * np.abs(R) + np.abs(ref_R - kw["alpha"] * R)
            within("R'", Ro, ref_R, E * size + (2 * U if self.res == torch.float32 else H) * np.abs(ref_R))
        if ref_H is None:
            assert Hh is None
        else:
            inv = 1 / np.sqrt((ref_R ** 2).mean(1, keepdims=True) + kw["eps"])
            # an error E size in R' also moves the mean square: at most E mean|size R'| / mean R'^2 of H
            moved = (size * np.abs(ref_R)).mean(1, keepdims=True) * inv ** 2
            tol = E * (np.abs(kw["w_pre"]) * inv * size + (1 + moved) * np.abs(ref_H))
            within("H", Hh, ref_H, tol + H * (np.abs(ref_H) + tol))
        return Ro, Hh

    def check_bwd(self, Ro=None, zero_dR=False):
        kw = self.params()
        M, C = self.R.shape
        p = self.norm
        Ro = self.R if Ro is None else Ro
        r, B = f64(Ro), None if self.B is None else f64(self.B)
        dR, dH = None if zero_dR else f64(self.dR), None if self.dH is None else f64(self.dH)
        ref = oracle.norm_bwd(r, B, dR, dH, **kw)
        got_dR, got_dB, grads = nf4.qlora_norm_bwd(p, Ro, self.B, None if zero_dR else self.dR, self.dH)
        assert set(grads) == {k for k, w in (("dw_pre", p.w_pre), ("dw_post", p.w_post), ("dgate", p.gate)) if w is not None}
        # sizes of t's terms
        t_size = np.zeros((M, C)) if dR is None else np.abs(dR)
        sums = (M + 32) * U
        if dH is not None:
            inv = 1 / np.sqrt((r ** 2).mean(1, keepdims=True) + kw["eps"])
            wd = np.abs(kw["w_pre"] * dH)
            t_size = t_size + inv * wd + np.abs(r) * inv ** 3 * (wd * np.abs(r)).mean(1, keepdims=True)
            size = (np.abs(dH) * np.abs(r) * inv).sum(0)
            within("dw_pre", grads["dw_pre"], ref["dw_pre"], H * np.abs(ref["dw_pre"]) + 1.01 * (E + sums) * size)
        res = 2 * U if self.res == torch.float32 else H
        within("dR", got_dR, ref["dR"], 1.01 * E * abs(kw["alpha"]) * t_size + res * np.abs(ref["dR"]))
        if B is None:
            assert got_dB is None
            return
        T = kw["gate_tokens"] or M
        g = np.ones((M, C)) if kw["gate"] is None else np.abs(kw["gate"])[np.arange(M) // T]
        u_size = abs(kw["beta"]) * g * t_size
        n = np.abs(B)
        b_size = u_size
        if p.w_post is not None:
            ib = 1 / np.sqrt((B ** 2).mean(1, keepdims=True) + kw["eps"])
            wu = np.abs(kw["w_post"]) * u_size
            n = np.abs(kw["w_post"]) * np.abs(B) * ib
            b_size = ib * wu + np.abs(B) * ib ** 3 * (wu * np.abs(B)).mean(1, keepdims=True)
            size = (u_size * np.abs(B) * ib).sum(0)
            within("dw_post", grads["dw_post"], ref["dw_post"], H * np.abs(ref["dw_post"]) + 1.01 * (2 * E + sums) * size)
        within("dB", got_dB, ref["dB"], H * np.abs(ref["dB"]) + 2.02 * E * b_size)
        if p.gate is not None:
            size = np.zeros(ref["dgate"].shape)
            np.add.at(size, np.arange(M) // T, abs(kw["beta"]) * t_size * n)
            within("dgate", grads["dgate"], ref["dgate"], H * np.abs(ref["dgate"]) + 1.01 * (2 * E + sums) * size)


SHAPES = [(1, 8), (3, 64), (2, 504), (5, 520), (4, 1024), (3, 1032), (7, 2048), (2, 2056), (4, 4096), (3, 4104), (2, 8192),
          (2, 8200), (1, 16384)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M,C", SHAPES)
def test_forward_and_backward_over_widths(M, C, f32):
    print(f"norm M={M} C={C} f32={f32}", flush=True)
    c = Case(M, C, gate=2, f32=f32, seed=M + C)
    if C <= 4104:
        c.check_bwd(c.check_fwd()[0])
    else:
        c.check_fwd()
        # the oracle forms C x C Jacobians: two rows at a time are enough
        c.check_bwd()


@pytest.mark.parametrize("pre,post,gate,f32", [(True, True, 0, False), (True, False, 0, True), (False, True, 0, False),
                                               (False, False, 1, False), (True, True, 1, True), (True, False, 3, False),
                                               (False, True, 40, True), (True, True, 1000, False), (True, False, 5, True)])
def test_parts_of_the_junction(pre, post, gate, f32):
    c = Case(41, 264, pre=pre, post=post, gate=gate, f32=f32, seed=3)
    c.check_bwd(c.check_fwd()[0])
    if pre:
        c.check_bwd(zero_dR=True)


@pytest.mark.parametrize("f32", [False, True])
def test_norm_before_a_block_alone(f32):
    c = Case(9, 520, post=False, f32=f32, block=False, seed=4)
    assert c.check_fwd()[0] is None
    c.check_bwd()
    c.check_bwd(zero_dR=True)


@pytest.mark.parametrize("M,gate", [(2500, 0), (2500, 1), (2500, 2), (2500, 3), (2500, 7), (2500, 600), (2500, 2499),
                                    (2500, 2500), (1030, 4), (4100, 5), (4100, 6)])
def test_many_rows_and_gate_runs(M, gate):
    """More rows than one run holds, gate rows shorter, longer and not a multiple of a run, a short last one."""
    c = Case(M, 64, gate=gate, seed=5)
    c.check_bwd(c.check_fwd()[0])


def test_no_gradients_of_the_weights():
    c = Case(33, 520, gate=4, seed=6)
    a = nf4.qlora_norm_bwd(c.norm, c.R, c.B, c.dR, c.dH)
    b = nf4.qlora_norm_bwd(c.norm, c.R, c.B, c.dR, c.dH, need_weights=False)
    assert b[2] == {} and same(a[0], b[0]) and same(a[1], b[1])


def test_rows_of_zeros_and_not_finite():
    c = Case(6, 520, gate=1, seed=7)
    clean = nf4.qlora_norm_fwd(c.norm, c.R, c.B, quantize=True)
    grads = nf4.qlora_norm_bwd(c.norm, clean[0], c.B, c.dR, c.dH)
    c.B[1] = 0
    c.R[1] = 0
    c.B[3, 7] = float("inf")
    c.R[4, 0] = float("nan")
    R, Hh, (q, s) = nf4.qlora_norm_fwd(c.norm, c.R, c.B, quantize=True)
    assert (R[1] == 0).all() and (Hh[1] == 0).all() and s[1] == 0 and (q[1] == 0).all()
    for m in (3, 4):
        assert not torch.isfinite(Hh[m]).all() and torch.isnan(s[m]) and (q[m] == 0).all()
    for m in (0, 2, 5):
        assert same(R[m], clean[0][m]) and same(Hh[m], clean[1][m]) and same(q[m], clean[2][0][m])
    dR, dB, _ = nf4.qlora_norm_bwd(c.norm, R, c.B, c.dR, c.dH)
    assert torch.isfinite(dR[1]).all() and torch.isfinite(dB[1]).all()      # eps keeps the zero row finite
    for m in (0, 2, 5):
        assert same(dR[m], grads[0][m]) and same(dB[m], grads[1][m])


@pytest.mark.parametrize("pre,f32", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("C", [520, 8200])
def test_tiny_rows_and_eps(C, pre, f32):
    """eps 1e-30, a row of zeros and one of about 1e-14: 1 / rms is up to 1e15 and its cube past float32."""
    c = Case(4, C, pre=pre, gate=2, f32=f32, seed=11)
    c.norm.eps = 1e-30
    c.R[0] = 0
    c.B[0] = 0
    c.R[2] *= 1e-14
    c.B[2] *= 1e-14
    c.check_fwd()
    c.check_bwd()


@pytest.mark.parametrize("C", [8, 512, 520, 2048, 4096, 8200, 16384])
@pytest.mark.parametrize("block", [False, True])
def test_codes_equal_those_of_h(C, block):
    c = Case(5, C, post=block, block=block, seed=8)
    out = nf4.qlora_norm_fwd(c.norm, c.R, c.B, quantize=True)
    plain = nf4.qlora_norm_fwd(c.norm, c.R, c.B)
    assert same(out[1], plain[1]) and (not block or same(out[0], plain[0]))
    q, s = nf4.nf4_int8_quantize(out[1])
    assert same(q, out[2][0]) and same(s, out[2][1])


@pytest.mark.parametrize("f32", [False, True])
def test_in_place_and_neighbours_untouched(f32):
    M, C = 37, 520
    c = Case(M, C, gate=5, f32=f32, seed=9)
    Ro, Hh = nf4.qlora_norm_fwd(c.norm, c.R, c.B)
    ref = nf4.qlora_norm_bwd(c.norm, Ro, c.B, c.dR, c.dH)

    def inside(t):
        b = torch.full((M + 2, C), 7.0, dtype=t.dtype, device=DEV)
        b[1:M + 1] = t
        return b, b[1:M + 1]

    bR, R = inside(c.R)
    bH, out_H = inside(torch.zeros_like(c.B))
    got = nf4.qlora_norm_fwd(c.norm, R, c.B, R_out=R, H=out_H)
    assert same(got[0], Ro) and same(got[1], Hh)
    bd, dR = inside(c.dR)
    bh, dH = inside(c.dH)
    got = nf4.qlora_norm_bwd(c.norm, Ro, c.B, dR, dH, dR=dR, dB=dH)
    assert same(got[0], ref[0]) and same(got[1], ref[1]) and all(same(got[2][k], ref[2][k]) for k in ref[2])
    for b in (bR, bH, bd, bh):
        assert (b[0] == 7).all() and (b[M + 1] == 7).all()


def test_repeats_bit_for_bit_with_a_dirty_workspace():
    for M, C, gate in ((700, 264, 0), (1500, 64, 100), (3000, 64, 2), (40, 8200, 7)):
        c = Case(M, C, gate=gate, seed=10)
        first = None
        for fill in (0, 0x7F, 0xFF):
            ws = torch.full((nf4.qlora_norm_workspace_size(M, C),), fill, dtype=torch.uint8, device=DEV)
            dR, dB, g = nf4.qlora_norm_bwd(c.norm, c.R, c.B, c.dR, c.dH, workspace=ws)
            out = [dR, dB] + [g[k] for k in sorted(g)]
            first = first or out
            assert all(same(a, b) for a, b in zip(first, out)), (M, C, fill)


@pytest.mark.parametrize("M,C,f32", [((1 << 21) + 9, 64, False), (600_005, 4096, False)])
def test_more_rows_than_a_launch_takes_and_offsets_past_32_bits(M, C, f32):
    """Rows do not know of each other: the last ones of a large call equal a small call's, bit for bit."""
    gate, last = 7, 7 * 5 + M % 7
    gen = torch.Generator(device=DEV)
    gen.manual_seed(M)
    n = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=DEV).normal_(0, 1, generator=gen)  # noqa: E731
    R, B, dR, dH = n(M, C), n(M, C), n(M, C), n(M, C)
    norm = nf4.QLoRANorm(w_pre=n(C), w_post=n(C), gate=n(-(-M // gate), C), gate_tokens=gate, alpha=0.5)
    tail = nf4.QLoRANorm(w_pre=norm.w_pre, w_post=norm.w_post, gate=norm.gate[(M - last) // gate:].contiguous(),
                         gate_tokens=gate, alpha=0.5)
    cut = lambda t: t[M - last:].contiguous()  # noqa: E731
    Ro, Hh, (q, s) = nf4.qlora_norm_fwd(norm, R, B, quantize=True)
    small = nf4.qlora_norm_fwd(tail, cut(R), cut(B), quantize=True)
    assert same(cut(Ro), small[0]) and same(cut(Hh), small[1]) and same(cut(q), small[2][0]) and same(cut(s), small[2][1])
    q2, s2 = nf4.nf4_int8_quantize(Hh)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    got_dR, got_dB, g = nf4.qlora_norm_bwd(norm, Ro, B, dR, dH)
    small_dR, small_dB, gs = nf4.qlora_norm_bwd(tail, small[0], cut(B), cut(dR), cut(dH))
    assert same(cut(got_dR), small_dR) and same(cut(got_dB), small_dB)
    # The two calls cut a gate row's tokens into runs differently, so its seven float32 terms are added in
    # another order: the sums differ by at most 2 * 6 u of the terms' sizes, and each is rounded to bf16
    # (h).  The terms' sizes from dR = alpha t (its own rounding, h, is the factor 1.01).
    b = f64(cut(B))
    n_size = np.abs(f64(norm.w_post) * b) / np.sqrt((b ** 2).mean(1, keepdims=True) + norm.eps)
    size = np.zeros(gs["dgate"].shape)
    np.add.at(size, np.arange(last) // gate, 1.01 * np.abs(f64(small_dR)) / 0.5 * n_size)
    ref = f64(gs["dgate"])
    within("dgate", g["dgate"][(M - last) // gate:], ref, 2 * H * 1.01 * np.abs(ref) + 12 * U * size)


def test_gradients_against_differences():
    """The whole junction through the kernels in float32 residuals: a small step of one input moves the
    loss by its gradient.  The loss sums R' (float32) only, so that no bf16 output hides the step."""
    c = Case(6, 64, pre=False, post=True, gate=2, f32=True, seed=11)
    Ro, _ = nf4.qlora_norm_fwd(c.norm, c.R, c.B)
    dR, dB, g = nf4.qlora_norm_bwd(c.norm, Ro, c.B, c.dR)
    loss = lambda: (nf4.qlora_norm_fwd(c.norm, c.R, c.B)[0].double() * c.dR.double()).sum().item()  # noqa: E731
    size = (Ro.double().abs() * c.dR.double().abs()).sum().item()
    for t, grad in ((c.R, dR), (c.B, dB), (c.norm.w_post, g["dw_post"]), (c.norm.gate, g["dgate"])):
        flat, gf = t.view(-1), grad.reshape(-1).double()
        for i in (0, 17, t.numel() - 1):
            x = flat[i].item()
            flat[i] = x + 0.0625 * max(abs(x), 0.25)
            hi, up = flat[i].item(), loss()
            flat[i] = x - 0.0625 * max(abs(x), 0.25)
            lo, down = flat[i].item(), loss()
            flat[i] = x
            # float32 rounding of R' (2 u of each term), the gradient's bf16 rounding, and the second
            # difference's third-order term: B and its rms only, at most (step / rms)^2 < 2^-3 / 64 of the row
            tol = 8 * U * size + abs(hi - lo) * (2 * H * abs(gf[i].item()) + 0.02)
            assert abs((up - down) - (hi - lo) * gf[i].item()) <= tol, (i, up - down, (hi - lo) * gf[i].item(), tol)


@pytest.mark.parametrize("M", [1, 300])
def test_captured_and_replayed(M):
    c = Case(M, 520, gate=7, seed=12)

    def step():
        R, Hh, q = nf4.qlora_norm_fwd(c.norm, c.R, c.B, quantize=True)
        dR, dB, g = nf4.qlora_norm_bwd(c.norm, R, c.B, c.dR, c.dH)
        return [R, Hh, q[0], q[1], dR, dB] + [g[k] for k in sorted(g)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for rep in range(3):
        new = Case(M, 520, gate=7, seed=20 + rep)
        for a, b in ((c.R, new.R), (c.B, new.B), (c.dR, new.dR), (c.dH, new.dH)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, step())), rep
        torch.cuda.synchronize()


def test_binding_refusals():
    c = Case(8, 64, gate=3, seed=13)
    p = c.norm
    for bad in (lambda: nf4.qlora_norm_fwd(p, c.R, c.B[:4]),
                lambda: nf4.qlora_norm_fwd(nf4.QLoRANorm(w_pre=p.w_pre[:32]), c.R),
                lambda: nf4.qlora_norm_fwd(nf4.QLoRANorm(w_pre=p.w_pre, gate=p.gate, gate_tokens=2), c.R, c.B),
                lambda: nf4.qlora_norm_fwd(nf4.QLoRANorm(w_pre=p.w_pre, gate=p.gate), c.R, c.B),
                lambda: nf4.qlora_norm_fwd(nf4.QLoRANorm(w_pre=p.w_pre), c.R, R_out=c.R),
                lambda: nf4.qlora_norm_fwd(nf4.QLoRANorm(w_post=p.w_post), c.R, c.B, quantize=True),
                lambda: nf4.qlora_norm_fwd(p, c.R[:, ::2], c.B),
                lambda: nf4.qlora_norm_bwd(p, c.R, c.B, c.dR[:3], c.dH)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        nf4.qlora_norm_fwd(p, c.R, c.B.float())
    for bad in (lambda: nf4.qlora_norm_fwd(p, c.R), lambda: nf4.qlora_norm_bwd(p, c.R, c.B, c.dR),
                lambda: nf4.qlora_norm_fwd(nf4.QLoRANorm(), c.R),
                lambda: nf4.qlora_norm_fwd(p, c.R[:0], c.B[:0]) if p.gate is None else nf4.qlora_norm_fwd(
                    nf4.QLoRANorm(w_pre=p.w_pre), c.R[:0])):
        with pytest.raises(nf4.NF4Error):
            bad()


def test_a_block_of_int8_linears_between_norms():
    """One gated MLP block as it is used: norm before (with codes), gate and up, SwiGLU, down, then norm
    after + gate + residual + the next norm; forward and backward, each stage against the oracle on the
    kernels' own inputs to it (relative Frobenius norm: a bf16 rounding each, 2^-8, and inner ones)."""
    M, C, F, r, s = 70, 320, 704, 8, 0.5
    c = Case(M, C, gate=16, f32=True, seed=14)
    before = nf4.QLoRANorm(w_pre=c.norm.w_post, eps=1e-5)
    n = lambda k, shape, std: torch.from_numpy(synth.normal_f32(8000 + k, shape, std)).to(DEV)  # noqa: E731
    lin = {}
    for i, (name, N, K) in enumerate((("gate", F, C), ("up", F, C), ("down", C, F))):
        lin[name] = (nf4.Int8Weight.from_float(n(3 * i, (N, K), 0.05)), n(3 * i + 1, (K, r), 1.0 / r).bfloat16(),
                     n(3 * i + 2, (r, N), 0.05).bfloat16())
    _, Hh, q = nf4.qlora_norm_fwd(before, c.R, quantize=True)
    G, Tg = nf4.qlora_int8_linear_fwd(lin["gate"][0], Hh, *lin["gate"][1:], s, Xq=q)
    Up, Tu = nf4.qlora_int8_linear_fwd(lin["up"][0], Hh, *lin["up"][1:], s, Xq=q)
    A = nf4.qlora_swiglu_fwd(G, Up)
    B, Td = nf4.qlora_int8_linear_fwd(lin["down"][0], A, *lin["down"][1:], s)
    R2, H2 = nf4.qlora_norm_fwd(c.norm, c.R, B)
    dR2, dB, gw = nf4.qlora_norm_bwd(c.norm, R2, B, c.dR, c.dH)
    dA, dL1d, dL2d = nf4.qlora_int8_linear_bwd(lin["down"][0], dB, A, *lin["down"][1:], Td, s)
    dG, dU = nf4.qlora_swiglu_bwd(dA, G, Up)
    dHh, dL1g, dL2g = nf4.qlora_int8_linear_bwd(lin["gate"][0], dG, Hh, *lin["gate"][1:], Tg, s)
    dHh, dL1u, dL2u = nf4.qlora_int8_linear_bwd(lin["up"][0], dU, Hh, *lin["up"][1:], Tu, s, dX=dHh, accumulate=True)
    dR, _, gb = nf4.qlora_norm_bwd(before, c.R, None, dR2, dHh)
    torch.cuda.synchronize()

    def near(name, got, ref, bound=oracle.REL_FRO_TOL):
        e = oracle.rel_fro(f64(got), ref)
        print(f"  {name}: {e:.2e}", flush=True)
        assert e <= bound, (name, e)

    eps = float(np.float32(1e-5))
    near("H", Hh, oracle.norm_fwd(f64(c.R), w_pre=f64(before.w_pre), eps=eps)[1])
    wb = {}
    for name, X, T, Y in (("gate", Hh, Tg, G), ("up", Hh, Tu, Up), ("down", A, Td, B)):
        w, L1, L2 = lin[name]
        Wq, ws = w.codes.cpu().numpy(), w.scales.cpu().numpy()
        wb[name] = oracle.bf16_to_f32(oracle.int8_weight_bf16(Wq, ws))
        near(name, Y, oracle.int8_product(*oracle.int8_rows(f64(X)), Wq, ws) + s * f64(X) @ f64(L1) @ f64(L2))
    near("A", A, oracle.swiglu_fwd(f64(G), f64(Up)))
    kw = c.params()
    ref_R, ref_H = oracle.norm_fwd(f64(c.R), f64(B), **kw)
    near("R'", R2, ref_R, 1e-5)
    near("H'", H2, ref_H)
    ref = oracle.norm_bwd(f64(R2), f64(B), f64(c.dR), f64(c.dH), **kw)
    near("dR'", dR2, ref["dR"], 1e-5)
    near("dB", dB, ref["dB"])
    for k in gw:
        near(k, gw[k], ref[k])
    ref = oracle.backward(f64(dB), f64(A), wb["down"], f64(lin["down"][1]), f64(lin["down"][2]), s)
    near("dA", dA, ref["dX"])
    near("dL1 down", dL1d, ref["dL1"])
    near("dL2 down", dL2d, ref["dL2"])
    rg, ru = oracle.swiglu_bwd(f64(dA), f64(G), f64(Up))
    near("dG", dG, rg)
    near("dU", dU, ru)
    a = oracle.backward(f64(dG), f64(Hh), wb["gate"], f64(lin["gate"][1]), f64(lin["gate"][2]), s)
    b = oracle.backward(f64(dU), f64(Hh), wb["up"], f64(lin["up"][1]), f64(lin["up"][2]), s)
    near("dH", dHh, a["dX"] + b["dX"])
    for name, got, want in (("dL1 gate", dL1g, a["dL1"]), ("dL2 gate", dL2g, a["dL2"]), ("dL1 up", dL1u, b["dL1"]),
                            ("dL2 up", dL2u, b["dL2"])):
        near(name, got, want)
    ref = oracle.norm_bwd(f64(c.R), None, f64(dR2), f64(dHh), w_pre=f64(before.w_pre), eps=eps)
    near("dR", dR, ref["dR"], 1e-5)
    near("dw", gb["dw_pre"], ref["dw_pre"])

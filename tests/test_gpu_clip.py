"""GPU parity of gradient clipping against the float64 oracle, and the end of a finetuning step: the loss's
gradient through a linear layer's backward into the clipped adapter gradients.

Tolerances (u = 2^-24, h = 2^-8): the norm is a float64 sum rounded to float32 once: u (and 1e-9 for the sum).  A clipped
element is a float64 product rounded to float32: u, then for bf16 that type's rounding (h on the rounded product).
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


def f64(t):
    return t.double().cpu().numpy()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def tensors(sizes, kinds, seed=0, std=1e-3):
    out = []
    for i, n in enumerate(sizes):
        t = torch.from_numpy(synth.normal_f32(8000 + 100 * seed + i, (n,), std)).to(DEV) if n else torch.empty(0, device=DEV)
        out.append(t.bfloat16() if kinds[i % len(kinds)] == "b" else t)
    return out


def check(grads, max_norm, outs=None):
    max_norm = float(np.float32(max_norm))       # the argument's type
    norm, ref = oracle.clip([f64(g) for g in grads], max_norm)
    before = [g.clone() for g in grads]
    got = nf4.qlora_clip_grads(nf4.QLoRAGrads(grads, outs), max_norm)
    assert got.shape == (1,) and got.dtype == torch.float32
    with np.errstate(over="ignore"):
        seen = float(np.float32(norm))
    assert float(got) == seen or abs(float(got) - norm) <= (U + 1e-9) * norm
    for b, g, o, r in zip(before, grads, outs or grads, ref):
        if outs is not None:
            assert same(b, g)
        if norm <= max_norm or np.isinf(seen):
            assert same(o, b)
        elif o.numel():
            tol = (H if o.dtype == torch.bfloat16 else 0.0) * np.abs(r) * (1 + U) + 1.01 * U * np.abs(r)
            tiny = 2.0 ** -133 if o.dtype == torch.bfloat16 else 2.0 ** -149       # half steps of the subnormals
            assert (np.abs(f64(o) - r) <= tol + tiny).all()
    return norm


SIZES = [1, 2, 3, 7, 8, 9, 63, 64, 65, 0, 1000, 4095, 4096, 4097, 8191, 8192, 8193, 20000, 5, 100001]


@pytest.mark.parametrize("kinds", ["b", "f", "bf", "fbb"])
@pytest.mark.parametrize("factor", [0.25, 0.999, 1.001, 50.0])
def test_lists(kinds, factor):
    grads = tensors(SIZES, kinds, seed=1)
    norm = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
    check([g.clone() for g in grads], norm / factor)
    check(grads, norm / factor, [torch.full_like(g, 9.0) for g in grads])


@pytest.mark.parametrize("n", [1, 95, 96, 97, 192, 193, 450])
def test_many_tensors(n):
    rng = np.random.default_rng(n)
    grads = tensors(rng.integers(0, 3000, n).tolist(), "bfb", seed=2)
    check(grads, 0.01)


def test_every_offset_and_guarded():
    """Tensors that begin and end anywhere in a buffer, gradient and output at different offsets."""
    for t, w in ((torch.bfloat16, 8), (torch.float32, 4)):
        for a in range(w + 1):
            for b in (0, 1, a, w - 1):
                for n in (1, w - 1, w, 3 * w + 1, 9000):
                    src = torch.full((n + 2 * w + 2,), 5.0, dtype=t, device=DEV)
                    dst = torch.full((n + 2 * w + 2,), 6.0, dtype=t, device=DEV)
                    g, o = src[a:a + n], dst[b:b + n]
                    g.copy_(torch.from_numpy(synth.normal_f32(77, (n,), 1.0)).to(DEV))
                    check([g], 0.5, [o])
                    assert (dst[:b] == 6).all() and (dst[b + n:] == 6).all()
                    check([g], 0.25)
                    assert (src[:a] == 5).all() and (src[a + n:] == 5).all()


def test_extreme_values():
    # squares past float32's range on both sides
    for v in (1e25, 1e-30):
        grads = [torch.full((100,), v, device=DEV), torch.full((33,), v, device=DEV).bfloat16()]
        check(grads, v)
    for t in (torch.float32, torch.bfloat16):
        check([torch.full((1000,), torch.finfo(t).max, dtype=t, device=DEV)], 1.0)
    # a norm past float32's range is not finite there; just inside, the factor is below that range
    check([torch.full((1000,), 1e36, device=DEV)], 1e-12)
    # a factor that sends values below the normal range
    check([torch.tensor([1.0, 2.0 ** -126, -(2.0 ** -140)], device=DEV)], 2.0 ** -9)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(bad):
    grads = tensors([1000, 33], "bf", seed=3)
    grads[1][7] = bad
    before = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    norm = nf4.qlora_clip_grads(nf4.QLoRAGrads(grads, outs), 1e-3)
    assert torch.isnan(norm).all() if np.isnan(bad) else float(norm) == np.inf
    nf4.qlora_clip_grads(nf4.QLoRAGrads(grads), 1e-3)
    for b, g, o in zip(before, grads, outs):
        assert same(b, g) and same(b, o)


def test_zeros_empty_and_norm_only():
    check([torch.zeros(100, device=DEV)], 1.0)
    assert float(nf4.qlora_clip_grads(nf4.QLoRAGrads([torch.empty(0, device=DEV)]), 1.0)) == 0.0
    grads = tensors([5000], "b", seed=4)
    check(grads, float("inf"))


def test_workspace_and_norm_given_other_stream_and_graph():
    grads = tensors([5000, 70001, 9], "bf", seed=5, std=1.0)
    outs = [torch.empty_like(g) for g in grads]
    lst = nf4.QLoRAGrads(grads, outs)
    assert len(lst) == 3 and lst.grads[0] is grads[0] and lst.outs[1] is outs[1]
    ref = nf4.qlora_clip_grads(lst, 1.0).clone()
    want = [o.clone() for o in outs]
    n = nf4.qlora_clip_workspace_size()
    ws = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    norm = torch.zeros(1, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            assert nf4.qlora_clip_grads(lst, 1.0, norm, ws) is norm
    s.synchronize()
    assert same(norm, ref) and all(same(a, b) for a, b in zip(outs, want)) and (ws[n:] == 0xA5).all()
    with pytest.raises(ValueError):
        nf4.qlora_clip_grads(lst, 1.0, norm, ws[:n - 1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nf4.qlora_clip_grads(lst, 1.0, norm, ws)
    for rep in range(3):
        for t in grads:
            t.mul_(0.5 + rep)
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        eager = nf4.qlora_clip_grads(lst, 1.0)
        torch.cuda.synchronize()
        assert same(eager, norm) and all(same(a, b) for a, b in zip(outs, got)), rep


def test_lists_are_checked():
    a, b = tensors([8, 16], "b", seed=6)
    for f in (lambda: nf4.QLoRAGrads([a, b[::2]]), lambda: nf4.QLoRAGrads([a], [b]), lambda: nf4.QLoRAGrads([a, b], [a])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: nf4.QLoRAGrads([a.double()]), lambda: nf4.QLoRAGrads([a], [a.float()]), lambda: nf4.QLoRAGrads([a.cpu()])):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(nf4.NF4Error):
        nf4.qlora_clip_grads(nf4.QLoRAGrads([a]), 0.0)


def test_end_of_a_finetuning_step():
    """Two NF4 linears with adapters, the head's loss on the responses only, back through both layers, and the four
    adapter gradients clipped: every stage against float64 arithmetic on that stage's own inputs."""
    M, K, N, V, r, s = 300, 256, 320, 1111, 16, 0.25
    t = lambda k, shape, std: torch.from_numpy(synth.normal_f32(8500 + k, shape, std)).to(DEV)  # noqa: E731
    w1, w2 = nf4.NF4Weight.from_float(t(0, (N, K), 0.05)), nf4.NF4Weight.from_float(t(1, (K, N), 0.05))
    ad = [t(2, (K, r), 0.1), t(3, (r, N), 0.1), t(4, (N, r), 0.1), t(5, (r, K), 0.1)]
    L1a, L2a, L1b, L2b = (a.bfloat16() for a in ad)
    X, head = t(6, (M, K), 1.0).bfloat16(), t(7, (V, K), 0.1).bfloat16()
    labels = torch.from_numpy(np.random.default_rng(1).integers(0, V, M)).to(DEV)
    labels[:180] = -100
    Y1, T1 = nf4.qlora_linear_fwd(w1, X, L1a, L2a, s)
    Y2, T2 = nf4.qlora_linear_fwd(w2, Y1, L1b, L2b, s)
    loss, mean, dY2 = nf4.qlora_loss_grad(head, Y2, labels)
    assert same(nf4.qlora_loss_fwd(head, Y2, labels)[0][:180], torch.zeros(180, device=DEV))
    ref, rmean, rd = oracle.loss(f64(Y2), f64(head), labels.cpu().numpy())
    assert oracle.within_tolerance(f64(dY2), rd) and abs(float(mean) - rmean) <= 1e-5 * rmean
    assert oracle.rel_fro(f64(loss), ref) <= 1e-5
    dY1, dL1b, dL2b = nf4.qlora_linear_bwd(w2, dY2, Y1, L1b, L2b, T2, s)
    _, dL1a, dL2a = nf4.qlora_linear_bwd(w1, dY1, X, L1a, L2a, T1, s, need_dX=False)
    g2 = oracle.backward(f64(dY2), f64(Y1), f64(nf4.nf4_dequant(w2)), f64(L1b), f64(L2b), s)
    assert oracle.within_tolerance(f64(dL1b), g2["dL1"]) and oracle.within_tolerance(f64(dY1), g2["dX"])
    assert not dY2[:180].any() and not dY1[:180].any()
    grads = [dL1a, dL2a, dL1b, dL2b]
    assert all(g.any() for g in grads)
    norm = check(grads, 1e-3)
    assert norm > 1e-3


def test_a_list_may_be_dropped_while_another_stream_still_reads_it():
    """The table's memory is not given out again before a call on another stream has ended (nothing is written to what is
    given out here)."""
    grads = tensors([5000, 70001, 9], "bf", seed=7, std=1.0)
    outs = [torch.empty_like(g) for g in grads]
    norm, ref = nf4.qlora_clip_grads(nf4.QLoRAGrads(grads, outs), 1.0), [o.clone() for o in outs]
    busy = torch.ones((8192, 8192), dtype=torch.bfloat16, device=DEV)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lst = nf4.QLoRAGrads(grads, outs)
    at, size = lst._table.data_ptr(), lst._table.numel()
    with torch.cuda.stream(s):
        for _ in range(40):
            busy = busy @ busy
        ended = torch.cuda.Event()
        got = nf4.qlora_clip_grads(lst, 1.0)
        ended.record()
    del lst
    new = [torch.empty(size, dtype=torch.int64, device=DEV) for _ in range(64)]
    waiting = not ended.query()
    assert waiting and at not in [t.data_ptr() for t in new]
    torch.cuda.synchronize()
    assert same(got, norm) and all(same(a, b) for a, b in zip(outs, ref))

"""The loss over the vocabulary and the clipping of gradients on the host: the oracle against differences and
closed forms, and every refusal of the entry points, before any HIP call."""
import ctypes

import numpy as np
import pytest

import oracle

nf4 = pytest.importorskip("bit_nf4_quantized_codebook_amd")
lib = nf4.lib

OK, ENULL, ESHAPE, EALIGN, EUNSUP, EWS, EHIP, EARG = 0, -1, -2, -3, -4, -5, -6, -7
FAKE = ctypes.c_void_p(0x100000)          # aligned, never dereferenced on these paths
MIS = ctypes.c_void_p(0x100004)
ODD = ctypes.c_void_p(0x100002)


# ---- the oracle against something other than itself ----

def test_loss_gradient_against_differences():
    rng = np.random.default_rng(11)
    M, V, K = 5, 9, 4
    X, W, g = rng.standard_normal((M, K)), rng.standard_normal((V, K)), rng.standard_normal(M)
    labels = np.array([3, -100, 0, 8, -1])
    each, mean, dX = oracle.loss(X, W, labels, g)
    assert not dX[[1, 4]].any() and each[1] == each[4] == 0
    assert abs(mean - each[[0, 2, 3]].sum() / 3) < 1e-15
    z = X @ W.T
    ref = np.log(np.exp(z).sum(1)) - z[np.arange(M), np.maximum(labels, 0)]
    assert np.allclose(each[[0, 2, 3]], ref[[0, 2, 3]], rtol=1e-13)
    dmean = oracle.loss(X, W, labels)[2]
    eps = 1e-6
    for m in range(M):
        for k in range(K):
            Xp, Xm = X.copy(), X.copy()
            Xp[m, k] += eps
            Xm[m, k] -= eps
            a, b = oracle.loss(Xp, W, labels), oracle.loss(Xm, W, labels)
            assert abs((a[0] @ g - b[0] @ g) / (2 * eps) - dX[m, k]) < 1e-8
            assert abs((a[1] - b[1]) / (2 * eps) - dmean[m, k]) < 1e-8


def test_loss_closed_forms():
    # equal logits: ln V; one entry: 0; a label ahead of V - 1 equal others by t: ln(1 + (V - 1) e^-t)
    assert abs(oracle.loss(np.zeros((1, 2)), np.ones((7, 2)), [2])[0][0] - np.log(7)) < 1e-15
    each, mean, dX = oracle.loss(np.ones((1, 2)), np.ones((1, 2)), [0])
    assert each[0] == 0 and mean == 0 and not dX.any()
    for t in (0.5, 30.0, 600.0, -40.0):
        W = np.zeros((5, 1))
        W[3] = t
        each, _, dX = oracle.loss(np.ones((1, 1)), W, [3], [1.0])
        ref = np.log1p(4 * np.exp(-t)) if t > 0 else np.log(4) - t + np.log1p(np.exp(t) / 4)
        assert abs(each[0] - ref) <= 1e-14 * ref
        assert abs(dX[0, 0] + t * 4 * np.exp(-t) / (1 + 4 * np.exp(-t))) <= 1e-12 * abs(t)
    each, mean, dX = oracle.loss(np.zeros((2, 1)), np.zeros((3, 1)), [-1, -7])
    assert mean == 0 and not each.any() and not dX.any()
    each, mean, dX = oracle.loss(np.zeros((2, 1)), np.zeros((3, 1)), [3, 1])
    assert np.isnan(each[0]) and np.isnan(dX[0]).all() and abs(each[1] - np.log(3)) < 1e-15


def test_clip_closed_forms():
    norm, out = oracle.clip([np.array([3.0]), np.array([[0.0, 4.0]])], 1.0)
    assert norm == 5.0 and abs(out[0][0] - 0.6) < 1e-15 and abs(out[1][0, 1] - 0.8) < 1e-15
    norm, out = oracle.clip([np.array([3.0, 4.0])], 5.0)
    assert norm == 5.0 and out[0].tolist() == [3.0, 4.0]
    norm, out = oracle.clip([np.array([np.inf, 1.0])], 1.0)
    assert norm == np.inf and out[0].tolist() == [np.inf, 1.0]


# ---- refusals ----

def test_loss_refusals():
    M, V, K = 8, 100, 128
    size = lib.qlora_loss_workspace_size
    wsf, wsg = size(M, V, K, 0), size(M, V, K, 1)
    assert 0 < wsf < wsg
    for bad in ((0, V, K), (-1, V, K), (M, 0, K), (M, V, 0), (M, V, 96), (M, V, 16448), ((1 << 20) + 1, V, 64),
                (M, (1 << 24) + 1, K), (1 << 20, V, 1024), (1 << 40, V, K)):
        assert size(*bad, 0) == 0 and size(*bad, 1) == 0, bad
    assert size(1 << 20, 1 << 24, 64, 0) > 0 and size(1, 1, 64, 1) > 0

    def fwd(W=FAKE, V=V, X=FAKE, labels=FAKE, M=M, K=K, loss=FAKE, mean=FAKE, ws=FAKE, n=wsf):
        return lib.qlora_loss_fwd(W, V, X, labels, M, K, loss, mean, ws, n, None)

    def grad(W=FAKE, V=V, X=FAKE, labels=FAKE, dloss=None, M=M, K=K, loss=FAKE, mean=FAKE, dX=FAKE, ws=FAKE, n=wsg):
        return lib.qlora_loss_grad(W, V, X, labels, dloss, M, K, loss, mean, dX, ws, n, None)

    for f, n in ((fwd, wsf), (grad, wsg)):
        assert f(M=0) == ESHAPE and f(M=-4) == ESHAPE and f(V=0) == ESHAPE and f(K=0) == ESHAPE and f(K=-64) == ESHAPE
        assert f(K=96) == EUNSUP and f(K=16448) == EUNSUP and f(M=(1 << 20) + 1) == EUNSUP and f(V=(1 << 24) + 1) == EUNSUP
        assert f(M=1 << 20, K=1024) == EUNSUP
        for k in ("W", "X", "labels", "loss", "mean"):
            assert f(**{k: None}) == ENULL, k
        assert f(W=MIS) == EALIGN and f(X=MIS) == EALIGN and f(labels=MIS) == EALIGN
        assert f(loss=ODD) == EALIGN and f(mean=ODD) == EALIGN and f(ws=MIS) == EALIGN
        assert f(ws=None) == EWS and f(n=n - 1) == EWS
    assert grad(dX=None) == ENULL and grad(dX=MIS) == EALIGN and grad(dloss=ODD) == EALIGN
    # dX over X, over the end of W, and ending inside X
    far, at = FAKE.value + (1 << 30), FAKE.value
    assert grad(W=far) == EARG and grad(X=far, dX=at + V * K * 2 - 16) == EARG and grad(W=far, dX=at - M * K * 2 + 16) == EARG


def test_loss_workspace_is_bounded_by_pieces():
    """The logits are never kept whole: beyond a piece of the vocabulary the workspace does not grow with it."""
    size = lib.qlora_loss_workspace_size
    M, K = 4096, 4096
    assert size(M, 1 << 20, K, 1) == size(M, 1 << 24, K, 1) < M * (1 << 20) * 2
    assert size(M, 1 << 20, K, 0) == size(M, 1 << 24, K, 0) < 1 << 27


def _grads(*entries):
    a = (nf4._GradDesc * max(len(entries), 1))()
    for i, e in enumerate(entries):
        a[i] = nf4._GradDesc(*e)
    return a


def test_grad_table_refusals():
    size = lib.qlora_grad_table_size
    assert size(-1) == 0 and size((1 << 20) + 1) == 0 and size(2) == 2 * size(1) == 2 * size(0)
    good = (0x100000, 0x100000, 10, 0)
    table, chunks = np.zeros(size(3) // 8, np.int64), ctypes.c_int64(-1)

    def make(*entries, n=None, null=False, at=0, bytes_=table.nbytes, out=True):
        a = _grads(*entries)
        return lib.qlora_grad_table(None if null else ctypes.addressof(a), len(entries) if n is None else n,
                                    None if at is None else table.ctypes.data + at, bytes_,
                                    ctypes.addressof(chunks) if out else None)

    assert make(good, n=-1) == ESHAPE and make(good, n=(1 << 20) + 1) == EUNSUP
    assert make(good, n=1, null=True) == ENULL and make(good, at=None) == ENULL and make(good, out=False) == ENULL
    assert make(good, at=4) == EALIGN and make(good, good, bytes_=size(2) - 1) == EWS
    assert make(good, (0x100000, 0x100000, 10, 2)) == EARG and make(good, (0x100000, 0x100000, -1, 0)) == ESHAPE
    assert make(good, (None, 0x100000, 1, 0)) == ENULL and make(good, (0x100000, None, 1, 0)) == ENULL
    assert make((0x100001, 0x100000, 1, 0)) == EALIGN and make((0x100000, 0x100001, 1, 0)) == EALIGN
    assert make((0x100002, 0x100000, 1, 1)) == EALIGN and make((0x100000, 0x100002, 1, 1)) == EALIGN
    assert make((0x100000, 0x100000, (1 << 46) + 1, 0)) == EUNSUP
    assert make(good, (0x100000, 0x100000, 1 << 46, 1)) == EUNSUP
    assert chunks.value == -1
    assert make((0x100002, 0x100104, 3, 0), (None, None, 0, 1), (0x200004, 0x200004, 1 << 30, 1)) == OK and chunks.value > 1
    assert make(null=True) == OK and chunks.value == 0


def test_grad_table_refuses_outputs_that_overlap():
    """Plain check of every pair of byte ranges against the table's answer, over lists of few, close tensors."""
    table, chunks = np.zeros(lib.qlora_grad_table_size(8) // 8, np.int64), ctypes.c_int64()

    def make(entries):
        a = _grads(*entries)
        return lib.qlora_grad_table(ctypes.addressof(a), len(entries), table.ctypes.data, table.nbytes, ctypes.addressof(chunks))

    def meet(a, b):
        return a[0] < b[1] and b[0] < a[1]

    def allowed(entries):
        full = [e for e in entries if e[2]]
        size = [e[2] * (4 if e[3] else 2) for e in full]
        g = [(e[0], e[0] + s) for e, s in zip(full, size)]
        o = [(e[1], e[1] + s) for e, s in zip(full, size)]
        pairs = [(i, j) for i in range(len(full)) for j in range(len(full)) if i != j]
        return (not any(meet(o[i], o[j]) or meet(o[i], g[j]) for i, j in pairs)
                and all(a == b or not meet(a, b) for a, b in zip(o, g)))

    rng = np.random.default_rng(3)
    seen = {OK: 0, EARG: 0}
    for _ in range(4000):
        entries = []
        for _ in range(int(rng.integers(1, 9))):
            g = 0x10000 + 16 * int(rng.integers(60))
            o = g if rng.integers(2) else 0x10000 + 8 * int(rng.integers(120))
            entries.append((g, o, int(rng.integers(0, 6)), int(rng.integers(2))))
        want = OK if allowed(entries) else EARG
        assert make(entries) == want, entries
        seen[want] += 1
    assert min(seen.values()) > 500, seen
    one = (0x1000, 0x1000, 8, 0)
    assert make([one, one]) == EARG                                                # scaled twice in place
    assert make([(0x1000, 0x2000, 8, 0), (0x1000, 0x3000, 8, 0)]) == OK            # counted twice, scaled to two places


def test_clip_refusals():
    wsb = lib.qlora_clip_workspace_size()

    def clip(table=FAKE, n=3, chunks=7, max_norm=1.0, norm=FAKE, ws=FAKE, size=wsb):
        return lib.qlora_clip_grads(table, n, chunks, max_norm, norm, ws, size, None)

    assert clip(n=-1) == ESHAPE and clip(chunks=-1) == ESHAPE and clip(n=0) == ESHAPE and clip(n=(1 << 20) + 1) == EUNSUP
    for bad in (0.0, -1.0, float("nan"), float("-inf")):
        assert clip(max_norm=bad) == EARG
    assert clip(table=None) == ENULL and clip(norm=None) == ENULL
    assert clip(table=MIS) == EALIGN and clip(norm=ODD) == EALIGN and clip(ws=MIS) == EALIGN
    assert clip(size=wsb - 1) == EWS and clip(ws=None) == EWS


def test_binding_refuses_host_tensors_and_empty_lists():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    lab = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: nf4.qlora_loss_fwd(x, x, lab), lambda: nf4.qlora_loss_grad(x, x, lab), lambda: nf4.QLoRAGrads([x]),
                 lambda: nf4.qlora_loss_fwd(x, None, lab), lambda: nf4.QLoRAGrads([None])):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: nf4.QLoRAGrads([]), lambda: nf4.QLoRAGrads([x], [x, x])):
        with pytest.raises(ValueError):
            call()


def test_a_list_on_another_stream_keeps_its_table(monkeypatch):
    """qlora_clip_grads tells the allocator of a stream that reads the list's table and is not the table's own."""
    torch = pytest.importorskip("torch")
    seen = []

    class Table:
        device = torch.device("cuda", 0)
        record_stream = staticmethod(seen.append)
        data_ptr = staticmethod(lambda: 0x1000)

    lst = nf4.QLoRAGrads.__new__(nf4.QLoRAGrads)
    lst._table, lst._grads, lst._outs, lst._chunks, lst._stream = Table(), (), (), 0, 11
    now = [11]
    monkeypatch.setattr(nf4, "_raw_stream", lambda index: now[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: ("stream", now[0]))
    monkeypatch.setattr(nf4, "_out", lambda t, dtype, shape, dev, name: torch.empty(shape))
    monkeypatch.setattr(nf4, "_scratch", lambda n, dev, ws: torch.empty(n, dtype=torch.uint8))
    calls = []
    monkeypatch.setattr(nf4, "_launch", lambda fn, name, dev, *a: calls.append(len(seen)))
    nf4.qlora_clip_grads(lst, 1.0)
    now[0] = 12
    nf4.qlora_clip_grads(lst, 1.0)
    assert seen == [("stream", 12)] and calls == [0, 1]


@pytest.mark.parametrize("M,MT", [(1, 64), (8, 64), (64, 64), (65, 128), (100, 128), (128, 128)])
def test_loss_workspace_of_few_tokens(M, MT):
    """A step of 64 vocabulary rows takes P for the 64 or 128 tokens of a tile, not 256, and three float32 a token; beside
    them stand dX's partials, which the vocabulary's length does not change from here on."""
    size, V, more, K = lib.qlora_loss_workspace_size, 64 * 512 * 8, 64 * 512, 64
    assert size(M, V + more, K, 1) - size(M, V, K, 1) <= 512 * (MT * 64 * 2 + 12 * M) + 4 * 256

"""GPU parity of the loss over the vocabulary (forward, and with its gradient) against the float64 oracle.

Tolerances, from the roundings on the way (u = 2^-24, h = 2^-8 for bf16).  A logit is a float32 sum of K exact
products in some order: off by at most Ez = K u sum |x w|.  In log2 units it is rounded again in one fma, so with the
constant's own error l - c is off by Ez / ln 2 + 4 u (|l| + |c|); 2^x in hardware adds 2 u, and a row's sum (64 in a
lane, then 4 across lanes and waves, then the tiles) at most (80 + tiles) u of itself.  With A = max |z| + 64 (c lies
within 48 of a maximum) every term of a row is off by the factor
  D = 2 (Ez + 8 u A) + (80 + tiles) u + 16 u,
d = ln S + c - z_label by D as well, and
  |loss error| <= sigmoid(d) D + 8 u loss,
  |dX error| <= |g| (sum_{v != y} p |W| (h + 2 D + V u) + (1 - p_y) |W_y| 2 D) (1 + h) + h |dX|.
Below float32's (and bf16's) smallest normal number, 2^-126, a value may be lost whole: a loss then is off by as much, and
dX, where 1 - p_y is such a value, by that times |sum p W / sum p - W_y| <= 2 max |W|, and its own rounding by 2^-126 again.
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
U, H, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -126
NONE = -100


def f64(t):
    return t.double().cpu().numpy()


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).bfloat16()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def make(M, V, K, seed=0, std=0.05, none=0.0, lift=0.0):
    rng = np.random.default_rng(100 + seed)
    X, W = synth.normal_f32(9000 + seed, (M, K), 1.0), synth.normal_f32(9500 + seed, (V, K), std)
    labels = rng.integers(0, V, M)
    W16 = f64(bf16(W))
    X = X + (lift * rng.random((M, 1)) * W16[labels] / np.maximum((W16[labels] ** 2).sum(1, keepdims=True), 1e-30)).astype(np.float32)
    labels[rng.random(M) < none] = NONE
    return bf16(X), bf16(W), torch.from_numpy(labels).to(DEV)


def check(X, W, labels, dloss=None, rows=None, fwd=True, grad=True):
    """Both entry points on these inputs, against the oracle at `rows` (all of them by default)."""
    M, K = X.shape
    V = W.shape[0]
    x, w, y = f64(X), f64(W), labels.cpu().numpy()
    rows = np.arange(M) if rows is None else rows
    count = int((y >= 0).sum())
    g = np.full(M, 1.0 / max(count, 1)) if dloss is None else f64(dloss)
    ref, _, dX = oracle.loss(x[rows], w, y[rows], g[rows])
    z = x[rows] @ w.T
    Ez = K * U * (np.abs(x[rows]) @ np.abs(w).T).max(1)
    tiles = -(-V // 256)
    D = 2 * (Ez + 8 * U * (np.abs(z).max(1) + 64)) + (96 + tiles) * U
    tol = -np.expm1(-ref) * D + 8 * U * ref + TINY
    out = []
    if fwd:
        out.append(nf4.qlora_loss_fwd(W, X, labels))
    if grad:
        out.append(nf4.qlora_loss_grad(W, X, labels, dloss))
    for o in out:
        got = f64(o[0])[rows]
        bad = ~(np.abs(got - ref) <= tol)
        assert not bad.any(), (int(bad.sum()), rows[bad][:5], got[bad][:5], ref[bad][:5], tol[bad][:5])
        assert not f64(o[0])[y < 0].any()
        assert abs(float(o[1]) - f64(o[0]).sum() / max(count, 1)) <= 2 * U * abs(float(o[1]))
    if grad:
        got = f64(out[-1][2])[rows]
        p = np.exp(z - (z[np.arange(len(rows)), np.maximum(y[rows], 0)] + ref)[:, None])
        p[np.arange(len(rows)), np.maximum(y[rows], 0)] = 0.0
        p[y[rows] < 0] = 0.0
        miss = -np.expm1(-ref)
        size = (p @ np.abs(w)) * (H + 2 * D + V * U)[:, None] + (miss * 2 * D)[:, None] * np.abs(w[np.maximum(y[rows], 0)])
        tolx = np.abs(g[rows])[:, None] * size * (1 + H) + H * np.abs(dX) + TINY * (1 + 2 * np.abs(w).max())
        bad = ~(np.abs(got - dX) <= tolx)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], dX[bad][:4], tolx[bad][:4])
        assert not f64(out[-1][2])[y < 0].any()
    return out


@pytest.mark.parametrize("M,V,K", [
    (1, 1, 64), (1, 2, 64), (3, 255, 64), (2, 256, 128), (5, 257, 64), (1, 1000, 512), (31, 300, 192), (64, 511, 64),
    (65, 513, 320), (255, 700, 64), (256, 256, 256), (257, 1025, 128), (300, 2049, 576), (513, 999, 1024),
    (4, 4099, 192), (16, 300, 64), (17, 4099, 192), (33, 16, 2048), (48, 129, 4160), (49, 30001, 64), (64, 15, 448), (128, 65, 192),
    (127, 64, 64), (128, 40000, 64), (100, 3000, 1984), (128, 7, 4096), (66, 641, 16384), (20, 129, 8256)])
def test_sizes(M, V, K):
    X, W, labels = make(M, V, K, seed=M + V, none=0.2 if M > 4 else 0.0, lift=12.0)
    check(X, W, labels)


@pytest.mark.parametrize("M", [129, 192, 256])
@pytest.mark.parametrize("none", [0.0, 0.4, 0.8])
@pytest.mark.parametrize("V,K", [(700, 320), (16384, 64), (16385, 64), (16500, 128), (32768, 64), (32769, 64), (300, 16384)])
def test_129_to_256_tokens(M, V, K, none):
    """Tiles for 64, 128 and 256 live tokens in one launch; one block of the vocabulary or two at a time, a last pair of
    one; the vocabulary from which tiles of 256 take over."""
    X, W, labels = make(M, V, K, seed=M + V, none=none, lift=10.0)
    labels[0], labels[-1] = V - 1, 0
    check(X, W, labels, torch.rand(M, device=DEV) - 0.3)


@pytest.mark.parametrize("M,none", [(256, 0.0), (200, 0.3), (200, 0.5), (130, 0.8)])
def test_references_move_within_pairs_of_blocks(M, none):
    """Logits of neighbouring blocks of 64 vocabulary rows far apart, either way round, and tokens that are not finite, a
    label past the vocabulary and tokens without one among them."""
    V, K = 16448 + 30, 64
    X, W, labels = make(M, V, K, seed=23, none=none)
    W[:, 0] = (torch.arange(V, device=DEV) // 64 % 5 * 9.0).bfloat16()
    X[:, 0] = torch.linspace(-7, 7, M, device=DEV).bfloat16()
    labels[1:4] = torch.tensor([5, 70, V - 1], device=DEV)
    check(X, W, labels, torch.ones(M, device=DEV))
    ref = nf4.qlora_loss_grad(W, X, labels, torch.ones(M, device=DEV))
    X[1, 3], labels[2] = float("nan"), V
    loss, mean, dX = nf4.qlora_loss_grad(W, X, labels, torch.ones(M, device=DEV))
    others = torch.ones(M, dtype=torch.bool, device=DEV)
    others[1:3] = False
    assert loss[1:3].isnan().all() and dX[1:3].isnan().all() and mean.isnan().all()
    assert same(loss[others], ref[0][others]) and same(dX[others], ref[2][others])


def test_graph_follows_the_number_of_live_tokens():
    M, V, K = 200, 16500, 128
    X, W, labels = make(M, V, K, seed=24)
    dX = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    loss, mean = torch.empty(M, device=DEV), torch.empty(1, device=DEV)
    ws = torch.empty(nf4.qlora_loss_workspace_size(M, V, K, True), dtype=torch.uint8, device=DEV)
    nf4.qlora_loss_grad(W, X, labels, None, loss, mean, dX, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nf4.qlora_loss_grad(W, X, labels, None, loss, mean, dX, ws)
    torch.cuda.synchronize()
    for live in (200, 40, 128, 0, 129, 64, 65, 1):
        lab = torch.full((M,), NONE, device=DEV, dtype=torch.int64)
        lab[torch.randperm(M, device=DEV)[:live]] = torch.randint(0, V, (live,), device=DEV)
        labels.copy_(lab)
        for t in (loss, mean, dX):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref = nf4.qlora_loss_grad(W, X, labels)
        torch.cuda.synchronize()
        for a, b in zip((loss, mean, dX), ref):
            assert same(a, b), live


@pytest.mark.parametrize("M", [60, 120, 600])
@pytest.mark.parametrize("none", [0.0, 0.5, 0.97, 1.0])
def test_tokens_without_a_label(none, M):
    X, W, labels = make(M, 777, 128, seed=3, none=none, lift=8.0)
    g = torch.rand(M, device=DEV) - 0.3
    check(X, W, labels, g)
    loss, mean, dX = nf4.qlora_loss_grad(W, X, labels)
    if none == 1.0:
        assert float(mean) == 0.0 and not dX.any() and not loss.any()
    # their X may hold anything; they are left as they are, whatever the others do
    X2 = X.clone()
    X2[labels < 0] = float("nan")
    again = nf4.qlora_loss_grad(W, X2, labels)
    assert same(again[0], loss) and same(again[1], mean) and same(again[2], dX)


@pytest.mark.parametrize("M", [65, 1024, 65536, 65537, 140001])
def test_live_rows_of_many_tokens(M):
    """Which rows take part, and in which order, over the runs that the list of live rows is made of."""
    V, K = 70, 64
    X, W, _ = make(64, V, K, seed=17)
    X = X[torch.arange(M, device=DEV) % 64].contiguous()          # 64 different tokens
    labels = torch.from_numpy(np.random.default_rng(M).integers(-V, V, M)).to(DEV)
    labels[200:400] = NONE
    labels[-1] = 5
    g = torch.rand(M, device=DEV)
    print(f"live rows: M={M} V={V} K={K}", flush=True)
    check(X, W, labels, g, rows=np.unique(np.concatenate([np.arange(min(M, 300)), np.arange(M - 65, M),
                                                          np.arange(max(0, min(M, 65536) - 70), min(M, 65606))])))


def test_any_negative_label_counts_as_none():
    X, W, labels = make(40, 300, 64, seed=5)
    a, b = labels.clone(), labels.clone()
    a[::3], b[::3] = NONE, torch.iinfo(torch.int64).min
    for p, q in zip(nf4.qlora_loss_grad(W, X, a), nf4.qlora_loss_grad(W, X, b)):
        assert same(p, q)


@pytest.mark.parametrize("M", [50, 100, 300])
def test_label_past_the_vocabulary_is_nan_alone(M):
    X, W, labels = make(M, 300, 64, seed=6)
    ref = nf4.qlora_loss_grad(W, X, labels, torch.ones(M, device=DEV))
    bad = labels.clone()
    bad[7], bad[41] = 300, torch.iinfo(torch.int64).max
    loss, mean, dX = nf4.qlora_loss_grad(W, X, bad, torch.ones(M, device=DEV))
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[[7, 41]] = False
    assert torch.isnan(loss[~keep]).all() and torch.isnan(dX[~keep]).all() and torch.isnan(mean).all()
    assert same(loss[keep], ref[0][keep]) and same(dX[keep], ref[2][keep])
    loss, mean = nf4.qlora_loss_fwd(W, X, bad)
    assert torch.isnan(loss[~keep]).all() and torch.isnan(mean).all() and torch.isfinite(loss[keep]).all()


@pytest.mark.parametrize("M", [40, 128, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_tokens_that_are_not_finite_stay_alone(value, M):
    X, W, labels = make(M, 700, 128, seed=7)
    g = torch.ones(M, device=DEV)
    ref = nf4.qlora_loss_grad(W, X, labels, g)
    X2, bad = X.clone(), M // 2 + 3
    X2[bad, 5] = value
    loss, mean, dX = nf4.qlora_loss_grad(W, X2, labels, g)
    keep = torch.arange(M, device=DEV) != bad
    assert torch.isnan(loss[bad]) and torch.isnan(dX[bad]).all() and torch.isnan(mean).all()
    assert same(loss[keep], ref[0][keep]) and same(dX[keep], ref[2][keep])


def test_sure_labels_keep_relative_accuracy():
    """Losses from 1e-30 up to hundreds: logits ahead of or behind the others by far."""
    M, V, K = 64, 600, 64
    X, W = np.zeros((M, K), np.float32), synth.normal_f32(31, (V, K), 0.05)
    W[:, 0] = 0.0
    labels = np.arange(M) * 9
    W[labels, 0] = 1.0                       # the label's logit moves with X[:, 0]
    others = np.setdiff1d(np.arange(V), labels)
    W[others, 0] = 0.0
    X[:] = synth.normal_f32(32, (M, K), 1.0)
    X[:, 0] = np.linspace(-250, 75, M)
    W[labels, 1:] = 0.0
    for m in range(M):                       # other tokens' label rows would answer too: one token a call
        w = W.copy()
        w[np.setdiff1d(labels, labels[m]), 0] = 0.0
        check(bf16(X[m:m + 1]), bf16(w), torch.tensor([labels[m]], device=DEV), torch.ones(1, device=DEV))


@pytest.mark.parametrize("M,V", [(3, 200), (12, 200), (20, 200), (100, 200), (200, 200), (200, 20000), (300, 200), (140, 33000)])
@pytest.mark.parametrize("above", [20.0, 64.0, 72.0])
def test_labels_far_above_the_reference(M, V, above):
    """The label's logit is e^94 and more, of which the references of the other entries, around e^30, know nothing."""
    X, W, labels = make(M, V, 64, seed=31)
    X[:, 0], W[:, 0] = 1.0, 30.0
    labels[:] = 7
    W[7, 0] = 30.0 + above
    check(X, W, labels, torch.ones(M, device=DEV))


@pytest.mark.parametrize("M", [1, 12, 30, 100, 200, 300])
@pytest.mark.parametrize("V", [1, 65, 193, 257, 2561])
def test_label_alone_in_its_tile(M, V):
    """The label is the last row of the vocabulary, alone in a tile of 16, 64 or 256, and all other logits lie far below a
    first reference of 0 (or above)."""
    for level, label in ((-150.0, -150.0), (-150.0, 40.0), (60.0, 60.0), (-40.0, 30.0)):
        X, W, labels = make(M, V, 64, seed=37)
        X[:, 0], W[:, 0], W[-1, 0] = 1.0, level, label
        labels[:] = V - 1
        check(X, W, labels, torch.ones(M, device=DEV))
        labels[:] = 0
        check(X, W, labels, torch.ones(M, device=DEV))


def test_references_move_far():
    """Each tile's largest logit exceeds the one before by more than a reference allows, up and down."""
    K, V = 64, 256 * 12
    for M, order in ((300, 1), (300, -1), (60, 1), (100, -1)):
        W = synth.normal_f32(41, (V, K), 0.05)
        W[:, 0] = np.repeat(np.arange(12)[::order] * 10.0, 256)
        X = synth.normal_f32(42, (M, K), 1.0)
        X[:, 0] = np.linspace(-6, 6, M)
        labels = np.random.default_rng(43).integers(0, V, M)
        check(bf16(X), bf16(W), torch.from_numpy(labels).to(DEV), torch.ones(M, device=DEV))


@pytest.mark.parametrize("order", [1, -1])
def test_pieces_of_the_vocabulary(order):
    """32768 tokens: a piece holds 8192 vocabulary rows, so three of them; the largest logits move from piece to
    piece.  Rows sampled."""
    M, V, K = 32768, 20001, 64
    assert nf4.qlora_loss_workspace_size(M, V, K, True) < 2 * M * V
    X, W, labels = make(M, V, K, seed=9, none=0.1, lift=10.0)
    W[:, 0] = (torch.arange(V, device=DEV) // 8192 * 9.0 * order).bfloat16()
    X[:, 0] = torch.linspace(-8, 8, M, device=DEV).bfloat16()
    rows = np.random.default_rng(10).choice(M, 150, replace=False)
    print(f"pieces: M={M} V={V} K={K} order={order}", flush=True)
    check(X, W, labels, rows=np.concatenate([rows, [0, M - 1]]))


@pytest.mark.parametrize("M", [60, 110, 130])
def test_outputs_and_workspace_given(M):
    V, K = 600, 128
    X, W, labels = make(M, V, K, seed=12, none=0.3)
    ref = nf4.qlora_loss_grad(W, X, labels)
    guard = torch.full((M + 2, K), 7.0, dtype=torch.bfloat16, device=DEV)
    loss, mean = torch.full((M + 2,), 7.0, device=DEV), torch.full((1,), 7.0, device=DEV)
    ws = torch.full((nf4.qlora_loss_workspace_size(M, V, K, True) + 64,), 0xA5, dtype=torch.uint8, device=DEV)
    out = nf4.qlora_loss_grad(W, X, labels, loss=loss[1:-1], mean=mean, dX=guard[1:-1], workspace=ws)
    for a, b in zip(out, ref):
        assert same(a, b)
    assert (guard[[0, -1]] == 7).all() and (loss[[0, -1]] == 7).all() and (ws[-64:] == 0xA5).all()
    out = nf4.qlora_loss_fwd(W, X, labels, loss=loss[1:-1], mean=mean, workspace=ws)
    assert out[1] is mean and (loss[[0, -1]] == 7).all()
    with pytest.raises(ValueError):
        nf4.qlora_loss_fwd(W, X, labels, workspace=ws[:64])


def test_refuses_what_does_not_fit():
    X, W, labels = make(8, 100, 64, seed=13)
    bad = [lambda: nf4.qlora_loss_fwd(W[:, :32], X, labels), lambda: nf4.qlora_loss_fwd(W.t(), X, labels),
           lambda: nf4.qlora_loss_fwd(W, X, labels[:-1]), lambda: nf4.qlora_loss_fwd(W, X[:, ::2], labels),
           lambda: nf4.qlora_loss_grad(W, X, labels, torch.ones(7, device=DEV)),
           lambda: nf4.qlora_loss_grad(W, X, labels, dX=torch.empty((8, 32), dtype=torch.bfloat16, device=DEV))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: nf4.qlora_loss_fwd(W.float(), X, labels), lambda: nf4.qlora_loss_fwd(W, X, labels.int()),
              lambda: nf4.qlora_loss_grad(W, X, labels, torch.ones(8, device=DEV).double())):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(nf4.NF4Error):
        nf4.qlora_loss_fwd(W[:, :32].contiguous(), X[:, :32].contiguous(), labels)


def test_gradient_against_differences_of_the_forward():
    """mean(X + D) - mean(X - D) = 2 <dX, D> up to a third of the third derivative along D.  That is the third central
    moment of (W D) under the token's softmax: at most 0.77 a^3 for values within [-a, a].  X and D are multiples of
    2^-6 below 4, so that X + D and X - D are exact in bf16."""
    M, V, K = 200, 3000, 256
    X, W, labels = make(M, V, K, seed=14, none=0.2, lift=6.0)
    X = (torch.round(X.float().clamp(-3.9, 3.9) * 64) / 64).bfloat16()
    _, _, dX = nf4.qlora_loss_grad(W, X, labels)
    D = torch.sign(dX.float()) / 64
    up, down = X.float() + D, X.float() - D
    assert (up.bfloat16().float() == up).all() and (down.bfloat16().float() == down).all()
    a, b = (nf4.qlora_loss_fwd(W, t.bfloat16(), labels)[1] for t in (up, down))
    live = labels >= 0
    count = int(live.sum())
    along = 2 * (dX.double() * D.double()).sum()
    moved = (D[live].double() @ W.double().t()).abs().max(1).values
    z = X[live].double() @ W.double().t()
    size = torch.softmax(z, 1) @ W.double().abs() + W[labels[live]].double().abs()
    tol = (0.77 * moved ** 3).sum() / 3 / count + 2 * H * (size * 2 / 64).sum() / count
    # both means are off by at most the logits' own error
    tol += 2 * K * U * (X.double().abs() @ W.double().abs().t()).max() * 2
    assert abs(float(a.double() - b.double()) - float(along)) <= float(tol)
    assert float(tol) < 0.1 * float(along)


@pytest.mark.parametrize("M", [33, 90, 400])
def test_other_stream_and_repeats(M):
    X, W, labels = make(M, 5000, 512, seed=15, none=0.3, lift=9.0)
    ref = nf4.qlora_loss_grad(W, X, labels)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        outs = [nf4.qlora_loss_grad(W, X, labels) for _ in range(3)]
    s.synchronize()
    for out in outs:
        for a, b in zip(out, ref):
            assert same(a, b)


@pytest.mark.parametrize("M", [50, 128, 300])
def test_graph_replays_match_eager(M):
    V, K = 2000, 256
    X, W, labels = make(M, V, K, seed=16, none=0.3)
    loss, mean = torch.empty(M, device=DEV), torch.empty(1, device=DEV)
    dX = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(nf4.qlora_loss_workspace_size(M, V, K, True), dtype=torch.uint8, device=DEV)
    nf4.qlora_loss_grad(W, X, labels, None, loss, mean, dX, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nf4.qlora_loss_grad(W, X, labels, None, loss, mean, dX, ws)
    torch.cuda.synchronize()
    for rep in range(3):
        X2, _, lab2 = make(M, V, K, seed=20 + rep, none=0.2 * rep)
        X.copy_(X2)
        labels.copy_(lab2)
        dX.fill_(float("nan"))
        loss.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        ref = nf4.qlora_loss_grad(W, X, labels)
        torch.cuda.synchronize()
        for a, b in zip((loss, mean, dX), ref):
            assert same(a, b), rep


@pytest.mark.parametrize("M,V,chain", [(1, 1500, 1500), (20, 1500, 1500), (100, 1500, 1500), (200, 1500, 1500),
                                       (200, 16500, 512), (300, 1500, 1500)])
def test_what_all_rows_have_in_common_cancels(M, V, chain):
    """A head whose rows share a part 40 times their own size in some columns, and tokens with one strong entry that is not
    the label.  With q the softmax without the label, w' = sum q W and 1 - p_y in front of it all, dX = sum q W - W_y.  P and
    the logits' errors are factors 1 + e on each q, |e| <= H + D, in the sum and in what divides it: that moves sum q W by
    sum q e (W - w') at most, without the common part.  Sums of at most `chain` terms are off by chain U of the sizes that go
    in (200 x 16500 x 128: parts of 5 steps of 64, 52 of them), the divisor by (104 + tiles) U."""
    K = 128
    X, W, labels = make(M, V, K, seed=51 + M + V, none=0.2 if M > 1 else 0.0)
    rng = np.random.default_rng(52)
    W = W.float()
    W[:, :32] += 2.0
    W = W.bfloat16()
    other = rng.integers(0, V, M)
    w16 = f64(W)
    own = w16[other].copy()
    own[:, :32] = 0.0                        # along the row's own part, to a share of about a half
    lift = (np.log(V) + 0.2 + rng.normal(0, 0.5, (M, 1))) * own / (own ** 2).sum(1, keepdims=True)
    x = f64(X)
    x[:, :32] /= 64.0
    X = bf16(x + lift)
    _, _, got = check(X, W, labels, torch.ones(M, device=DEV), fwd=False)[0]
    x, y, tiles = f64(X), labels.cpu().numpy(), -(-V // 256)
    _, _, ref = oracle.loss(x, w16, y, np.ones(M))
    D = 2 * (K * U * (np.abs(x) @ np.abs(w16).T).max(1) + 8 * U * (np.abs(x @ w16.T).max(1) + 64)) + (96 + tiles) * U
    for m in np.flatnonzero(y >= 0):
        z = w16 @ x[m]
        q = np.exp(z - np.delete(z, y[m]).max())
        miss = (q.sum() - q[y[m]]) / q.sum()
        q[y[m]] = 0.0
        q /= q.sum()
        mid = q @ w16
        size = (H * (1 + 2 * H) + 2 * D[m]) * (q @ np.abs(w16 - mid)) + chain * U * (q @ np.abs(w16)) \
            + (104 + tiles) * U * np.abs(mid) + 4 * U * np.abs(w16[y[m]])
        tol = miss * size * (1 + H) + (2 * D[m] + H) * np.abs(ref[m]) + TINY
        err = np.abs(f64(got[m]) - ref[m])
        assert (err <= tol).all(), (m, int((err > tol).sum()), float((err / tol).max()))


@pytest.mark.parametrize("M", [1, 3, 12, 40, 100, 200, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_weight_rows_that_are_not_finite(value, M):
    """One value of W: every token meets its row.  A logit that is NaN or +inf, or the label's own if it is not finite, gives
    NaN; another row's -inf is a probability of zero, which leaves the loss finite and dX NaN in that value's column alone.
    The finite ones against the oracle: D as at the top, of the other rows, which are as they were."""
    V, K, row, col = 700, 128, 333, 5
    X, W, labels = make(M, V, K, seed=61 + M, none=0.2 if M > 20 else 0.0)
    labels[::3] = row
    x, y, g = f64(X), labels.cpu().numpy(), torch.ones(M, device=DEV)
    w = f64(W)
    D = 2 * (K * U * (np.abs(x) @ np.abs(w).T).max(1) + 8 * U * (np.abs(x @ w.T).max(1) + 64)) + (96 + 3) * U
    W[row, col] = w[row, col] = value
    with np.errstate(invalid="ignore", over="ignore"):
        ref, rmean, rdX = oracle.loss(x, w, y, np.ones(M))
    down = (y >= 0) & (y != row) & (value * x[:, col] == -np.inf)
    assert (np.isfinite(ref) == (down | (y < 0))).all()
    loss, mean, dX = nf4.qlora_loss_grad(W, X, labels, g)
    for each, m in ((loss, mean), nf4.qlora_loss_fwd(W, X, labels)):
        got = f64(each)
        assert (np.isnan(got) == np.isnan(ref)).all()
        ok = np.isfinite(ref)
        assert (np.abs(got - ref)[ok] <= (D + 8 * U * ref + TINY)[ok]).all()
        assert np.isnan(float(m)) == np.isnan(rmean)
    got = f64(dX)
    assert np.isnan(got[np.isnan(ref)]).all() and not got[y < 0].any()
    assert np.isnan(got[down, col]).all() and np.isfinite(np.delete(got[down], col, 1)).all()
    keep = np.arange(K) != col
    size = 2 * np.abs(w[np.arange(V) != row]).max()          # of |sum q W - W_y|, of which 1 + e on each q moves H + 2 D
    assert (np.abs(got - rdX)[down][:, keep] <= ((H + 2 * D)[down, None] + V * U) * size + H * np.abs(rdX[down][:, keep])).all()


def check_sampled(X, W, labels, dloss, rows):
    """check() for large W: the definition in float64 on the device, 4096 vocabulary rows at a time, at `rows` (with a label)."""
    M, K = X.shape
    V = W.shape[0]
    at = torch.as_tensor(rows, device=DEV)
    x, y, g = X[at].double(), labels[at], dloss[at].double()
    assert (y >= 0).all()
    blocks = [slice(i, min(i + 4096, V)) for i in range(0, V, 4096)]

    def dots(a, f):
        return torch.cat([a @ f(W[b].double()).t().contiguous() for b in blocks], 1)

    z = dots(x, lambda w: w)
    Ez = K * U * dots(x.abs(), torch.abs).max(1).values
    D = (2 * (Ez + 8 * U * (z.abs().max(1).values + 64)) + (96 + -(-V // 256)) * U)[:, None]
    rest = z - z.gather(1, y[:, None])
    rest.scatter_(1, y[:, None], -float("inf"))
    d = torch.logsumexp(rest, 1, keepdim=True)
    ref = torch.clamp(d, min=0) + torch.log1p(torch.exp(-d.abs()))
    p, miss, wy = torch.exp(rest - ref), torch.sigmoid(d), W[y].double()
    pw, size = torch.zeros_like(wy), torch.zeros_like(wy)
    for b in blocks:
        w = W[b].double()
        pw += p[:, b].contiguous() @ w
        size += p[:, b].contiguous() @ w.abs()
    dX = g[:, None] * (pw - miss * wy)
    tol = miss * D + 8 * U * ref + TINY
    tolx = g[:, None].abs() * (size * (H + 2 * D + V * U) + miss * 2 * D * wy.abs()) * (1 + H) + H * dX.abs() \
        + TINY * (1 + 2 * float(W.abs().max()))
    out = nf4.qlora_loss_fwd(W, X, labels), nf4.qlora_loss_grad(W, X, labels, dloss)
    for o in out:
        err = (o[0][at].double() - ref[:, 0]).abs() / tol[:, 0]
        assert (err <= 1).all(), float(err.max())
        each = o[0].double()
        assert not o[0][labels < 0].any() and abs(float(o[1]) - float(each.sum() / (labels >= 0).sum())) <= 2 * U * abs(float(o[1]))
    err = (out[1][2][at].double() - dX).abs() / tolx
    assert (err <= 1).all(), (float(err.max()), torch.nonzero(~(err <= 1))[:4].tolist())
    assert not out[1][2][labels < 0].any()


def some(labels, n, seed=0):
    """n of the tokens with a label, the first and the last among them."""
    live = torch.nonzero(labels >= 0)[:, 0].cpu().numpy()
    return np.unique(np.concatenate([live[[0, -1]], np.random.default_rng(seed).choice(live, min(n, len(live)), replace=False)]))


def in_pieces(M, V, K, grad):
    """The vocabulary is not taken in one piece: twice as many rows need no more workspace."""
    assert nf4.qlora_loss_workspace_size(M, V, K, grad) == nf4.qlora_loss_workspace_size(M, 2 * V, K, grad)


@pytest.mark.parametrize("M,V,K,none", [(300, 69888, 256, 0.0), (700, 8000, 8192, 0.0), (1200, 8000, 8192, 0.45),
                                        (1700, 14000, 4096, 0.0)])
def test_tails_of_parts_in_runs(M, V, K, none):
    """Tiles of dX beyond whole rounds whose parts leave tails, shared by runs of the workgroups left over: a run inside a tile
    (2 tiles), and runs that begin in one tile and end in another (96 and 112)."""
    X, W, labels = make(M, V, K, seed=71, none=none, lift=9.0)
    print(f"runs: M={M} V={V} K={K}", flush=True)
    check_sampled(X, W, labels, torch.rand(M, device=DEV) + 0.1, some(labels, 60))


@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("M,none", [(8192, 0.0), (8300, 0.0), (9000, 0.08)])
def test_pieces_added_by_the_product(M, none, order):
    """Pieces of the vocabulary with 256 tiles of dX and more, whose sums the product itself adds to what the piece before
    left; the largest logits move from piece to piece, and the row's reference with them."""
    V, K = 33000, 2048
    in_pieces(M, V, K, True)
    X, W, labels = make(M, V, K, seed=72, none=none, lift=8.0)
    W[:, 0] = (torch.arange(V, device=DEV) // 8192 * 9.0 * order).bfloat16()
    X[:, 0] = torch.linspace(-8, 8, M, device=DEV).bfloat16()
    print(f"pieces: M={M} V={V} K={K} order={order}", flush=True)
    check_sampled(X, W, labels, torch.rand(M, device=DEV) + 0.1, some(labels, 60))


@pytest.mark.parametrize("order", [1, -1])
def test_forward_in_pieces(order):
    """65537 tokens: the forward's tables hold 63 tiles of 256 vocabulary rows, and there are 65."""
    M, V, K = 65537, 16400, 64
    in_pieces(M, V, K, False)
    X, W, labels = make(64, V, K, seed=73, lift=8.0)
    W[:, 0] = (torch.arange(V, device=DEV) // 4100 * 9.0 * order).bfloat16()
    X = X[torch.arange(M, device=DEV) % 64].contiguous()
    X[:, 0] = torch.linspace(-8, 8, M, device=DEV).bfloat16()
    labels = labels[torch.arange(M, device=DEV) % 64].contiguous()
    labels[::7] = NONE
    print(f"forward pieces: M={M} V={V} K={K} order={order}", flush=True)
    check_sampled(X, W, labels, torch.rand(M, device=DEV) + 0.1, some(labels, 100))


@pytest.mark.parametrize("M", [8, 100])
def test_few_tokens_where_the_weight_exceeds_2_gib(M):
    """The gradient then takes W in two pieces, and with them the large tiles; up to 8 tokens the sums' one workgroup writes
    the mean."""
    V, K = 65700, 16384
    in_pieces(M, V, K, True)
    g = torch.Generator(device=DEV)
    g.manual_seed(74)
    W = torch.randn((V, K), generator=g, device=DEV, dtype=torch.bfloat16).mul_(0.02)
    W[:, 0] = (torch.arange(V, device=DEV) // 65280 * 6.0).bfloat16()
    X = torch.randn((M, K), generator=g, device=DEV, dtype=torch.bfloat16)
    X[:, 0] = torch.linspace(-3, 3, M, device=DEV).bfloat16()
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    labels[0], labels[1], labels[2] = V - 1, 65279, NONE
    print(f"W of 2 GiB: M={M} V={V} K={K}", flush=True)
    check_sampled(X, W, labels, torch.rand(M, device=DEV) + 0.1, some(labels, 60))


def far_logits(M, V, K, seed, size):
    """Logits of about 8 `size`; returns also float64 logits, and D's logit part: how far off one may be (natural units)."""
    X, W, labels = make(M, V, K, seed=seed, none=0.2 if M > 4 else 0.0)
    X, W = (X.float() * size).bfloat16(), (W.float() * 20.0).bfloat16()
    x, w = X.double(), W.double().t().contiguous()
    z = x @ w
    off = K * U * (x.abs() @ w.abs()).max(1).values + 8 * U * (z.abs().max(1).values + 64)
    return X, W, labels, z, off


@pytest.mark.parametrize("M,V,K", [(1, 700, 64), (3, 20, 64), (12, 700, 64), (40, 700, 128), (100, 700, 64), (200, 700, 64), (200, 17000, 64),
                                   (300, 700, 64), (32768, 20001, 64)])
@pytest.mark.parametrize("size", [2.0 ** 20, 1e9, 1e14, 1e30])
def test_logits_beyond_what_a_reference_resolves(M, V, K, size):
    """Logits so large that neighbouring float32 values are hundreds apart and more: a token's softmax then is its largest
    logit alone, wherever that exceeds the next by far more than the logits' own error (their error E, twice and 100 more)."""
    X, W, labels, z, off = far_logits(M, V, K, 81 + M + V, size)
    g = torch.ones(M, device=DEV)
    out = nf4.qlora_loss_fwd(W, X, labels), nf4.qlora_loss_grad(W, X, labels, g)
    y = labels.clamp(min=0)
    zl = z.gather(1, y[:, None])[:, 0]
    z.scatter_(1, y[:, None], -float("inf"))
    top, at = z.topk(2, 1)
    d = top[:, 0] - zl
    clear = (labels >= 0) & (top[:, 0] - top[:, 1] > 2 * off + 100) & (d.abs() > 2 * off + 100)
    assert clear.any()
    ref = torch.clamp(d, min=0)
    for o in out:
        assert not o[0][labels < 0].any()
        err = (o[0].double() - ref).abs()[clear]
        assert (err <= (2 * off + 8 * U * ref)[clear]).all(), (int((err > (2 * off + 8 * U * ref)[clear]).sum()), float(err.max()))
    # its probability is 1 but for e^-100, and so is 1 - p_y, or e^-100 at most where the label is ahead
    want = torch.where(d[:, None] > 0, W[at[:, 0]].double() - W[y].double(), 0.0)
    most = W.double().abs().max()
    assert ((out[1][2].double() - want).abs()[clear] <= (H * want.abs() + 4 * U * most + TINY)[clear]).all()


@pytest.mark.parametrize("M,V,K", [(1 << 20, 300, 64), (65535, 300, 16384), (1, 1 << 24, 64), (16, 1 << 24, 64), (24, 1 << 24, 64)])
def test_largest_sizes(M, V, K):
    """The most tokens, an X just below 2 GiB, and the most vocabulary rows (W of 2 GiB)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(91)
    X = torch.randn((M, K), generator=g, device=DEV, dtype=torch.bfloat16)
    W = torch.randn((V, K), generator=g, device=DEV, dtype=torch.bfloat16).mul_(0.05)
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    labels[-1] = V - 1
    if M > 16:
        labels[::5] = NONE
        labels[0] = 0
    print(f"largest: M={M} V={V} K={K}", flush=True)
    check_sampled(X, W, labels, torch.rand(M, device=DEV) + 0.1, some(labels, 40))

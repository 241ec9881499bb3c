"""Measured cases of the two ends of a finetuning step: the loss over the vocabulary and the clipping
of the adapters' gradients.

Three operators, each in its plain form (elementary torch operations) and through the package:

* loss_fwd   softmax cross entropy of the output head, logits = X W^T with W [V, K] frozen: the loss
             of each token and their mean over the tokens that have a label (evaluation, perplexity);
* loss_grad  the same with the gradient of the mean, or of weighted losses, with respect to X (the
             training step; tokens without a label, such as a prompt's, have loss and gradient zero);
* clip       the global norm of many gradient tensors, and all of them scaled down to a largest norm.

Sizes are those of this repository's workloads (LLaMA-7B and 65B widths, their adapters at rank 64;
a vocabulary of 32000) and generic ones, ragged ones among them.
"""
import math

import torch

own = False

DEV = "cuda"
IGNORE = -100


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def _loss(op, M, V, K, ignored=0.0, weighted=False):
    """ignored: the part of the tokens without a label; weighted: a gradient of its own for each token's
    loss in place of the mean's."""
    case = {"op": op, "M": M, "V": V, "K": K, "ignored": ignored}
    return {**case, "weighted": weighted} if op == "loss_grad" else case


def _clip(kind, n, width, r, size):
    """kind: "bf16", "f32" or "mixed"; n adapter pairs [width, r] and [r, width']; size: the gradient's
    norm over the largest allowed norm."""
    return {"op": "clip", "kind": kind, "n": n, "width": width, "r": r, "size": size}


def listed():
    return [
        # the answer token of a multiple-choice question, 7B width
        {"name": "loss_fwd_1x32000x4096", **_loss("loss_fwd", 1, 32000, 4096)},
        # a few short answers scored together, an odd vocabulary
        {"name": "loss_fwd_37x50001x4096", **_loss("loss_fwd", 37, 50001, 4096)},
        # perplexity of a ragged text over a large odd vocabulary
        {"name": "loss_fwd_511x131071x4096", **_loss("loss_fwd", 511, 131071, 4096)},
        # perplexity of a full context at the 65B width
        {"name": "loss_fwd_2048x32000x8192", **_loss("loss_fwd", 2048, 32000, 8192)},
        # the training step of a small micro-batch: a prompt with a short response
        {"name": "loss_grad_129x32000x4096", **_loss("loss_grad", 129, 32000, 4096, 0.7)},
        # a ragged micro-batch at the 65B width, a weight for each token, an odd vocabulary
        {"name": "loss_grad_777x50001x8192", **_loss("loss_grad", 777, 50001, 8192, 0.1, True)},
        # the 7B training step, every token with a label
        {"name": "loss_grad_4096x32000x4096", **_loss("loss_grad", 4096, 32000, 4096)},
        # the same where only the responses have labels
        {"name": "loss_grad_4096x32000x4096_responses", **_loss("loss_grad", 4096, 32000, 4096, 0.6)},
        # two sequences of 4096 tokens over a large vocabulary
        {"name": "loss_grad_8192x131072x4096", **_loss("loss_grad", 8192, 131072, 4096)},
        # the adapter of one 7B projection
        {"name": "clip_one_pair_4096_bf16", **_clip("bf16", 1, 4096, 64, 2.5)},
        # the adapters on every linear of 32 layers at the 7B width
        {"name": "clip_224_pairs_4096_bf16", **_clip("bf16", 224, 4096, 64, 1.7)},
        # ragged adapters with gradients in both types, as a program that accumulates some in float32 has them
        {"name": "clip_61_pairs_5003_mixed", **_clip("mixed", 61, 5003, 24, 30.0)},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step if int(v) >= step else step))


def draw(rng):
    op = rng.choice(["loss_fwd", "loss_fwd", "loss_grad", "loss_grad", "clip"])
    if op == "clip":
        n, r = _log(rng, 1, 224), rng.choice([8, 16, 24, 64])
        width = _log(rng, 256, min(8192, (224 * 2048 * 64) // (n * r)))
        return _clip(rng.choice(["bf16", "f32", "mixed"]), n, width, r, rng.choice([0.3, 1.5, 40.0]))
    V, K = _log(rng, 1000, 131072), _log(rng, 512, 8192, 64)
    M = _log(rng, 1, min(8192, (8192 * 131072 * 4096) // (V * K)))
    return _loss(op, M, V, K, rng.choice([0.0, 0.25, 0.6, 0.9]), rng.random() < 0.4)


def _counted(c):
    """Tokens with a label."""
    return c["M"] - int(c["ignored"] * c["M"])


def _clip_shapes(c):
    """(shape, type) of every gradient: the pairs' second widths follow a decoder layer's seven linears
    (two of the MLP's width, 43/16 of the model's)."""
    wide = c["width"] * 43 // 16
    out = []
    for i in range(c["n"]):
        a, b = [(c["width"], c["width"])] * 4 + [(c["width"], wide)] * 2 + [(wide, c["width"])], i % 7
        k, n = a[b]
        f32 = c["kind"] == "f32" or (c["kind"] == "mixed" and i % 3 == 1)
        t = torch.float32 if f32 else torch.bfloat16
        out += [((k, c["r"]), t), ((c["r"], n), t)]
    return out


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device=DEV) * std


def prepare(case, seed):
    c, s = dict(case), {"case": dict(case)}
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["op"] == "clip":
        # the gradients lie one after the other in a bucket for each type, as an all-reduce takes them
        shapes = _clip_shapes(c)
        s["buckets"], total = {}, 0.0
        for t in dict.fromkeys(t for _, t in shapes):
            n = sum(shape[0] * shape[1] for shape, of in shapes if of == t)
            x = _normal(g, (n,), 1e-3)
            # a gradient in twenty is a hundred times the others
            x = torch.where(torch.rand((n,), generator=g, device=DEV) < 0.05, x * 100.0, x).to(t)
            s["buckets"][t] = (x, torch.empty_like(x))
            total += float(x.double().square().sum())
        s["max_norm"] = math.sqrt(total) / c["size"]
        s["grads"], s["out"], at = [], [], dict.fromkeys(s["buckets"], 0)
        for shape, t in shapes:
            n = shape[0] * shape[1]
            for name, bucket in zip(("grads", "out"), s["buckets"][t]):
                s[name].append(bucket[at[t]:at[t] + n].view(shape))
            at[t] += n
        return s
    M, V, K = c["M"], c["V"], c["K"]
    w = _normal(g, (V, K), 0.02).bfloat16()
    labels = torch.randint(0, V, (M,), generator=g, device=DEV)
    # hidden states after the last norm: unit normals with a few strong channels, and a part along the
    # label's row that raises its logit by 0 to 20, from tokens missed to tokens known for sure
    x = _normal(g, (M, K), 1.0)
    x[:, int(torch.randint(0, min(K, 256), (1,), generator=g, device=DEV))::256] *= 3.0
    up = torch.rand((M, 1), generator=g, device=DEV) * 20.0
    wl = w[labels].float()
    x += up * wl / wl.square().sum(1, keepdim=True)
    none = int(c["ignored"] * M)
    labels[torch.randperm(M, generator=g, device=DEV)[:none]] = IGNORE
    s.update(W=w, X=x.bfloat16(), labels=labels)
    if c["op"] == "loss_grad":
        s["dloss"] = torch.rand(M, generator=g, device=DEV) * (2.0 / M) if c["weighted"] else None
    return s


# ------------------------------------------------------------------------------------------
# plain forms, in 32 bits
# ------------------------------------------------------------------------------------------

def _plain_loss(s):
    c = s["case"]
    live = (s["labels"] >= 0).nonzero()[:, 0]
    label = s["labels"][live][:, None]
    w = s["W"].float()
    z = s["X"][live].float() @ w.t()
    zl = z.gather(1, label)
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    # the others' sum by itself: log(sum e^z) - z_label cancels where the label is nearly certain
    rest = e.scatter(1, label, 0.0).sum(1, keepdim=True)
    d = torch.log(rest) + m - zl
    each = torch.clamp(d, min=0.0) + torch.log1p(torch.exp(-d.abs()))
    loss = torch.zeros(c["M"], device=DEV)
    loss[live] = each[:, 0]
    out = {"loss": loss, "mean": (each.double().sum() / each.numel()).float().reshape(1)}
    if c["op"] == "loss_fwd":
        return out
    p = e / (rest + torch.exp(zl - m))
    p.scatter_(1, label, -1.0 / (1.0 + torch.exp(-d)))
    p *= s["dloss"][live][:, None] if s["dloss"] is not None else 1.0 / each.numel()
    dX = torch.zeros((c["M"], c["K"]), dtype=torch.bfloat16, device=DEV)
    dX[live] = (p @ w).bfloat16()
    return {**out, "dX": dX}


def _plain_clip(s):
    total = torch.stack([(x.float() * x.float()).sum() for x in s["grads"]]).double().sum()
    norm = torch.sqrt(total).float()
    factor = torch.clamp(s["max_norm"] / norm, max=1.0)
    for x, y in zip(s["grads"], s["out"]):
        y.copy_(x.float() * factor)
    return {"norm": norm.reshape(1), "grads": [y for _, y in s["buckets"].values()]}


# ------------------------------------------------------------------------------------------
# the package's calls
# ------------------------------------------------------------------------------------------

def _own_run(s):
    import bit_nf4_quantized_codebook_amd as nf4
    op = s["case"]["op"]
    if op == "clip":
        if "list" not in s:
            s["list"] = nf4.QLoRAGrads(s["grads"], s["out"])
        norm = nf4.qlora_clip_grads(s["list"], s["max_norm"])
        return {"norm": norm, "grads": [y for _, y in s["buckets"].values()]}
    if op == "loss_fwd":
        loss, mean = nf4.qlora_loss_fwd(s["W"], s["X"], s["labels"])
        return {"loss": loss, "mean": mean}
    loss, mean, dX = nf4.qlora_loss_grad(s["W"], s["X"], s["labels"], s["dloss"])
    return {"loss": loss, "mean": mean, "dX": dX}


def run(state):
    if own:
        return _own_run(state)
    return _plain_clip(state) if state["case"]["op"] == "clip" else _plain_loss(state)


def work(case):
    c = case
    if c["op"] == "clip":
        n = size = 0
        for shape, t in _clip_shapes(c):
            k = shape[0] * shape[1]
            n, size = n + k, size + k * (4 if t == torch.float32 else 2)
        return {"bytes": 2 * size + 4, "flops": 3 * n}
    # the tokens without a label take no part in the products
    M, V, K, live = c["M"], c["V"], c["K"], _counted(c)
    fwd = {"bytes": 2 * V * K + 2 * live * K + 12 * M, "flops": 2 * live * V * K + 4 * live * V}
    if c["op"] == "loss_fwd":
        return fwd
    return {"bytes": fwd["bytes"] + 2 * M * K + (4 * M if c["weighted"] else 0), "flops": 2 * fwd["flops"]}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "clip":
        buckets = [x.double() for x, _ in s["buckets"].values()]
        norm = math.sqrt(math.fsum(float(torch.dot(x, x)) for x in buckets))
        scale = min(1.0, s["max_norm"] / norm)
        return {"norm": torch.tensor([norm], dtype=torch.float64, device=DEV), "grads": [x * scale for x in buckets]}
    M, V, K = c["M"], c["V"], c["K"]
    labels, counted = s["labels"], _counted(c)
    loss = torch.zeros(M, dtype=torch.float64, device=DEV)
    dX = torch.zeros((M, K), dtype=torch.float64, device=DEV) if c["op"] == "loss_grad" else None
    w64 = s["W"].double()
    w64t = w64.t().contiguous()
    # rows at a time: a block of logits of about 2 GB
    step = max(1, (1 << 28) // V)
    for i in range(0, M, step):
        lab = labels[i:i + step]
        ok = lab >= 0
        at = lab.clamp(min=0).unsqueeze(1)
        logits = torch.mm(s["X"][i:i + step].double(), w64t)
        target = logits.gather(1, at)
        # against the label's own logit: loss = log(1 + sum over the others of exp(z_v - z_label))
        logits.sub_(target).scatter_(1, at, float("-inf"))
        top = logits.max(dim=1, keepdim=True).values
        others = torch.exp(logits - top).sum(dim=1, keepdim=True)
        gap = (others.log() + top)[:, 0]
        value = torch.where(gap > 0, gap + torch.log1p(torch.exp(-gap)), torch.log1p(torch.exp(gap)))
        loss[i:i + step] = torch.where(ok, value, torch.zeros_like(value))
        if dX is not None:
            prob = torch.exp(logits - value.unsqueeze(1))
            prob.scatter_(1, at, -torch.sigmoid(gap).unsqueeze(1))
            weight = s["dloss"][i:i + step].double() if s["dloss"] is not None else torch.full_like(value, 1.0 / counted)
            prob *= torch.where(ok, weight, torch.zeros_like(weight)).unsqueeze(1)
            dX[i:i + step] = torch.mm(prob, w64)
    out = {"loss": loss, "mean": (loss.sum() / counted).reshape(1)}
    return out if dX is None else {**out, "dX": dX}

"""Measured cases of the Int8 linear layer and of the norm glue between blocks.

Four operators, each in its plain form (elementary torch operations) and through the package:

* quantize   rows to 8-bit integers with one constant per row (activations by token, weights by
             output channel);
* linear     Y = sx sw (Xq Wq^T) + s (X L1) L2, forward ("fwd") and backward ("bwd");
* norm_fwd   R' = alpha R + beta gate * norm(B; w_post), H = norm(R'; w_pre);
* norm_bwd   its backward.

Sizes are those of this repository's workloads (LLaMA-7B and 65B-shaped linears, the 28672 x 8192
decode weight) and ragged ones of the same ranges.
"""
import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def _quant(rows, cols, f32):
    return {"op": "quantize", "rows": rows, "cols": cols, "f32": f32}


def _linear(op, M, N, K, r):
    return {"op": op, "M": M, "N": N, "K": K, "r": r}


def _norm(op, M, C, post, gate_tokens, f32):
    return {"op": op, "M": M, "C": C, "post": post, "gate_tokens": gate_tokens, "f32": f32}


def listed():
    return [
        # a float32 weight of the 7B MLP quantized when a model is loaded
        {"name": "quantize_weight_f32_11008x4096", **_quant(11008, 4096, True)},
        # activations of a short ragged prompt before a linear
        {"name": "quantize_tokens_bf16_777x8192", **_quant(777, 8192, False)},
        # one decoded token through the large decode weight, with its adapter
        {"name": "linear_fwd_decode_1x28672x8192", **_linear("linear_fwd", 1, 28672, 8192, 64)},
        # a small serving batch on the 7B down projection, adapters merged
        {"name": "linear_fwd_batch_23x4096x11008", **_linear("linear_fwd", 23, 4096, 11008, 0)},
        # a training step's tokens through a 7B attention projection
        {"name": "linear_fwd_4096x4096x4096", **_linear("linear_fwd", 4096, 4096, 4096, 64)},
        # the 65B-shaped gate projection
        {"name": "linear_fwd_2048x22016x8192", **_linear("linear_fwd", 2048, 22016, 8192, 64)},
        # backward of the 7B attention projection
        {"name": "linear_bwd_4096x4096x4096", **_linear("linear_bwd", 4096, 4096, 4096, 64)},
        # backward of a ragged small batch with a narrow adapter through the 7B up projection
        {"name": "linear_bwd_333x11008x4096", **_linear("linear_bwd", 333, 11008, 4096, 16)},
        # between two blocks while decoding one token
        {"name": "norm_fwd_decode_1x8192", **_norm("norm_fwd", 1, 8192, True, 1, False)},
        # between two blocks of a training step: residual kept in float32, one gate for all tokens
        {"name": "norm_fwd_4096x4096_f32", **_norm("norm_fwd", 4096, 4096, True, 4096, True)},
        # backward of the same in bf16, one gate row per sequence of 512 tokens
        {"name": "norm_bwd_4096x4096", **_norm("norm_bwd", 4096, 4096, True, 512, False)},
        # backward of a plain pre-norm residual block, ragged tokens, wide rows
        {"name": "norm_bwd_1001x8192_f32", **_norm("norm_bwd", 1001, 8192, False, 0, True)},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step if int(v) >= step else step))


def draw(rng):
    op = rng.choice(["quantize", "linear_fwd", "linear_fwd", "linear_bwd", "norm_fwd", "norm_bwd"])
    if op == "quantize":
        cols = _log(rng, 64, 28672, 8)
        rows = _log(rng, 1, min(32768, (1 << 28) // cols))
        return _quant(rows, cols, rng.random() < 0.5)
    if op.startswith("linear"):
        N, K = _log(rng, 256, 28672, 8), _log(rng, 256, 22016, 64)
        most = min(4096, max(1, (2048 * 22016 * 8192 // (1 if op == "linear_fwd" else 2)) // (N * K)))
        M = _log(rng, 1, most)
        return _linear(op, M, N, K, rng.choice([0, 8, 16, 64, 128]))
    C = _log(rng, 256, 16384, 8)
    M = _log(rng, 1, min(8192, (1 << 25) // C))
    post = rng.random() < 0.6
    gate = rng.choice([0, 1, M, _log(rng, 1, M)])
    return _norm(op, M, C, post, gate, rng.random() < 0.5)


def _gate_rows(c):
    return -(-c["M"] // c["gate_tokens"]) if c["gate_tokens"] else 0


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device=DEV) * std


def _activations(g, M, K):
    """Hidden states: unit normals, with one channel in 256 twenty times as large."""
    x = _normal(g, (M, K), 1.0)
    x[:, int(torch.randint(0, min(K, 256), (1,), generator=g, device=DEV))::256] *= 20.0
    return x.bfloat16()


def _weight_f32(g, N, K):
    """Weights: normals of standard deviation 0.02, one in a hundred ten times as large."""
    w = _normal(g, (N, K), 0.02)
    return torch.where(torch.rand((N, K), generator=g, device=DEV) < 0.01, w * 10.0, w)


def prepare(case, seed):
    c, s = dict(case), {"case": dict(case)}
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if c["op"] == "quantize":
        s["X"] = _weight_f32(g, c["rows"], c["cols"]) if c["f32"] else _activations(g, c["rows"], c["cols"])
        return s
    if c["op"].startswith("linear"):
        M, N, K, r = c["M"], c["N"], c["K"], c["r"]
        s["Wq"], s["Ws"] = _codes(_weight_f32(g, N, K))
        s["X"] = _activations(g, M, K)
        s["scale"] = 16.0 / r if r else 1.0
        s["L1"] = _normal(g, (K, r), 1.0 / r).bfloat16() if r else None
        s["L2"] = _normal(g, (r, N), 0.01).bfloat16() if r else None
        if c["op"] == "linear_bwd":
            s["dY"] = _normal(g, (M, N), 1.0).bfloat16()
            s["T"] = (s["X"].float() @ s["L1"].float()).bfloat16() if r else None
        return s
    M, C = c["M"], c["C"]
    like = torch.float32 if c["f32"] else torch.bfloat16
    s["R"] = _normal(g, (M, C), 2.0).to(like)
    s["B"] = _normal(g, (M, C), 0.7).bfloat16()
    s["w_pre"] = (1.0 + _normal(g, (C,), 0.1)).bfloat16()
    s["w_post"] = (1.0 + _normal(g, (C,), 0.1)).bfloat16() if c["post"] else None
    s["gate"] = (0.5 + _normal(g, (_gate_rows(c), C), 0.2)).bfloat16() if c["gate_tokens"] else None
    s["alpha"], s["beta"] = 0.9375, 0.25
    if c["op"] == "norm_bwd":
        s["dR"] = _normal(g, (M, C), 1.0).to(like)
        s["dH"] = _normal(g, (M, C), 1.0).bfloat16()
    return s


# ------------------------------------------------------------------------------------------
# plain forms: 32 bits throughout; a code's quotient in 64, since a value next to the border
# between two codes may not fall on the other side
# ------------------------------------------------------------------------------------------

def _codes(x):
    absmax = x.abs().amax(1).double()
    scale = (absmax / 127.0).float()
    per = torch.where(scale > 0, scale, torch.ones_like(scale)).double()
    return torch.round(x.double() / per[:, None]).clamp(-127, 127).to(torch.int8), scale


def _plain_linear_fwd(s):
    xq, xs = _codes(s["X"].float())
    y = (xq.float() @ s["Wq"].float().t()) * xs[:, None] * s["Ws"][None, :]
    if s["L1"] is None:
        return {"Y": y.bfloat16()}
    t = s["X"].float() @ s["L1"].float()
    return {"Y": (y + s["scale"] * (t @ s["L2"].float())).bfloat16(), "T": t.bfloat16()}


def _plain_linear_bwd(s):
    # the gradient runs through the weight in bf16, the layer's compute type
    w = (s["Wq"].float() * s["Ws"][:, None]).bfloat16().float()
    dy = s["dY"].float()
    dx = dy @ w
    if s["L1"] is None:
        return {"dX": dx.bfloat16()}
    dt = s["scale"] * (dy @ s["L2"].float().t())
    return {"dX": (dx + dt @ s["L1"].float().t()).bfloat16(), "dL1": (s["X"].float().t() @ dt).bfloat16(),
            "dL2": (s["scale"] * (s["T"].float().t() @ dy)).bfloat16()}


def _gate_of(s, like):
    """The gate's row for each token, or 1."""
    c = s["case"]
    if s["gate"] is None:
        return 1.0
    return s["gate"].to(like).repeat_interleave(c["gate_tokens"], 0)[: c["M"]]


def _plain_norm_fwd(s):
    b = s["B"].float()
    n = b * torch.rsqrt(b.square().mean(1, keepdim=True) + EPS) * s["w_post"].float() if s["w_post"] is not None else b
    r = s["alpha"] * s["R"].float() + s["beta"] * _gate_of(s, torch.float32) * n
    h = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * s["w_pre"].float()
    return {"R": r.to(s["R"].dtype), "H": h.bfloat16()}


def _plain_norm_bwd(s):
    c = s["case"]
    # R holds the residual after the block, as the forward wrote it
    r, b, dh = s["R"].float(), s["B"].float(), s["dH"].float()
    inv_r = torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
    xh, wd = r * inv_r, s["w_pre"].float() * dh
    t = s["dR"].float() + inv_r * (wd - xh * (wd * xh).mean(1, keepdim=True))
    out = {"dR": (s["alpha"] * t).to(s["R"].dtype), "dw_pre": (dh * xh).sum(0).bfloat16()}
    n = b
    if s["w_post"] is not None:
        inv_b = torch.rsqrt(b.square().mean(1, keepdim=True) + EPS)
        bh = b * inv_b
        n = bh * s["w_post"].float()
    if s["gate"] is not None:
        each = s["beta"] * t * n
        whole = torch.zeros((_gate_rows(c) * c["gate_tokens"], c["C"]), device=each.device)
        whole[: c["M"]] = each
        out["dgate"] = whole.view(-1, c["gate_tokens"], c["C"]).sum(1).bfloat16()
    u = s["beta"] * _gate_of(s, torch.float32) * t
    if s["w_post"] is None:
        return {**out, "dB": u.bfloat16()}
    wu = s["w_post"].float() * u
    db = inv_b * (wu - bh * (wu * bh).mean(1, keepdim=True))
    return {**out, "dB": db.bfloat16(), "dw_post": (u * bh).sum(0).bfloat16()}


# ------------------------------------------------------------------------------------------
# the package's calls
# ------------------------------------------------------------------------------------------

def _own_run(s):
    import bit_nf4_quantized_codebook_amd as nf4
    op = s["case"]["op"]
    if op == "quantize":
        codes, scales = nf4.nf4_int8_quantize(s["X"])
        return {"codes": codes, "scales": scales}
    if op.startswith("linear"):
        if "w" not in s:
            s["w"] = nf4.Int8Weight(s["Wq"], s["Ws"])
        if op == "linear_fwd":
            Y, T = nf4.qlora_int8_linear_fwd(s["w"], s["X"], s["L1"], s["L2"], s["scale"])
            return {"Y": Y} if T is None else {"Y": Y, "T": T}
        dX, dL1, dL2 = nf4.qlora_int8_linear_bwd(s["w"], s["dY"], s["X"], s["L1"], s["L2"], s["T"], s["scale"])
        return {"dX": dX} if dL1 is None else {"dX": dX, "dL1": dL1, "dL2": dL2}
    if "norm" not in s:
        s["norm"] = nf4.QLoRANorm(w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"],
                                  gate_tokens=s["case"]["gate_tokens"], alpha=s["alpha"], beta=s["beta"], eps=EPS)
    if op == "norm_fwd":
        R, H = nf4.qlora_norm_fwd(s["norm"], s["R"], s["B"])
        return {"R": R, "H": H}
    dR, dB, grads = nf4.qlora_norm_bwd(s["norm"], s["R"], s["B"], s["dR"], s["dH"])
    return {"dR": dR, "dB": dB, **grads}


def run(state):
    if own:
        return _own_run(state)
    op = state["case"]["op"]
    if op == "quantize":
        codes, scales = _codes(state["X"].float())
        return {"codes": codes, "scales": scales}
    return {"linear_fwd": _plain_linear_fwd, "linear_bwd": _plain_linear_bwd,
            "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd}[op](state)


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (5 if c["f32"] else 3) + 4 * c["rows"], "flops": 3 * n}
    if c["op"].startswith("linear"):
        M, N, K, r = c["M"], c["N"], c["K"], c["r"]
        weights = N * K + 4 * N + 2 * r * (K + N)
        if c["op"] == "linear_fwd":
            return {"bytes": weights + 2 * M * (K + N + r), "flops": 2 * M * N * K + 2 * M * r * (K + N)}
        adapters = 2 * M * K + 2 * M * r + 2 * r * (K + N) if r else 0
        return {"bytes": weights + 2 * M * N + 2 * M * K + adapters,
                "flops": 2 * M * N * K + 4 * M * r * (K + N)}
    M, C, res = c["M"], c["C"], 4 if c["f32"] else 2
    vectors = 2 * C * (1 + (1 if c["post"] else 0) + _gate_rows(c))
    if c["op"] == "norm_fwd":
        return {"bytes": M * C * (2 * res + 4) + vectors, "flops": 12 * M * C}
    return {"bytes": M * C * (3 * res + 6) + 2 * vectors, "flops": 30 * M * C}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------

def _rows64(x):
    """Values that the rows' 8-bit codes stand for: (codes, constants), in float64."""
    x = x.double()
    step = (x.abs().max(dim=1).values / 127).to(torch.float32).double()
    q = torch.zeros_like(x)
    live = step > 0
    q[live] = torch.round(x[live] / step[live].unsqueeze(1)).clamp(min=-127, max=127)
    return q, step


def _inv_rms64(x):
    return 1.0 / torch.sqrt((x * x).sum(1) / x.shape[1] + EPS)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantize":
        q, step = _rows64(s["X"])
        return {"codes": q.to(torch.int8), "scales": step}
    if c["op"].startswith("linear"):
        wq, ws, x = s["Wq"].double(), s["Ws"].double(), s["X"].double()
        l1, l2 = (None, None) if s["L1"] is None else (s["L1"].double(), s["L2"].double())
        if c["op"] == "linear_fwd":
            q, step = _rows64(s["X"])
            y = torch.mm(q * step.unsqueeze(1), (wq * ws.unsqueeze(1)).t().contiguous())
            if l1 is None:
                return {"Y": y}
            t = torch.mm(x, l1)
            return {"Y": y.add_(torch.mm(t, l2), alpha=s["scale"]), "T": t}
        # the weight of the backward is defined as its bf16 value
        w = (wq * ws.unsqueeze(1)).float().bfloat16().double()
        dy = s["dY"].double()
        dx = torch.mm(dy, w)
        if l1 is None:
            return {"dX": dx}
        dt = torch.mm(dy, l2.t().contiguous()) * s["scale"]
        return {"dX": dx + torch.mm(dt, l1.t().contiguous()), "dL1": torch.mm(x.t().contiguous(), dt),
                "dL2": torch.mm(s["T"].double().t().contiguous(), dy) * s["scale"]}
    M, C = c["M"], c["C"]
    token = torch.arange(M, device=DEV)
    gate = s["gate"].double()[token // c["gate_tokens"]] if s["gate"] is not None else torch.ones((M, C), dtype=torch.float64, device=DEV)
    b, r, wp = s["B"].double(), s["R"].double(), s["w_pre"].double()
    ib = _inv_rms64(b).unsqueeze(1)
    post = s["w_post"].double() if c["post"] else None
    n = b if post is None else b * ib * post
    if c["op"] == "norm_fwd":
        r = s["alpha"] * r + s["beta"] * (gate * n)
        return {"R": r, "H": wp * (r * _inv_rms64(r).unsqueeze(1))}
    # derivative of y = w x / sqrt(mean x^2 + eps): inv (w dy) - x inv^3 <w dy, x> / C
    ir, dh = _inv_rms64(r).unsqueeze(1), s["dH"].double()
    along = ((wp * dh) * r).sum(1, keepdim=True) / C
    t = s["dR"].double() + ir * (wp * dh) - r * (ir ** 3) * along
    out = {"dR": s["alpha"] * t, "dw_pre": (dh * (r * ir)).sum(0)}
    u = s["beta"] * gate * t
    if s["gate"] is not None:
        out["dgate"] = torch.zeros((_gate_rows(c), C), dtype=torch.float64, device=DEV).index_add_(
            0, token // c["gate_tokens"], s["beta"] * t * n)
    if post is None:
        return {**out, "dB": u}
    along = (post * u * b).sum(1, keepdim=True) / C
    return {**out, "dB": ib * post * u - b * (ib ** 3) * along, "dw_post": (u * (b * ib)).sum(0)}

"""The operators around an 8-bit product, as cases to be measured: RMS norm with the
residual's addition and an 8-bit output, its gradient, the int8 product with a scale
for each token and channel, and the log probabilities of given tokens with their
entropy and top alternatives, and their gradient.

A case is a dict of plain values; ``op`` names the operator.  ``run`` computes it by
elementary torch operations in 32 bits, or, with ``own`` true, through this package.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ES = {"bf16": 2, "f16": 2, "f32": 4}
_QT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "int8": torch.int8}
_QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}
_EPS = 1e-6
_IGNORE = -100
_SCALE_MIN = 2.0 ** -126

# the most that one drawn case may need, per operator (bytes moved; products)
_NORM_BYTES = 8192 * 5760 * 7
_GRAD_BYTES = 8192 * 5760 * 8
_INT8_PRODUCTS = 8192 * 5760 * 1920
_LOGIT_BYTES = 4095 * 131072 * 2
_LOGIT_GRAD_BYTES = 2047 * 50001 * 2 * 2


def listed():
    return [
        # one new token entering a decode step's FP8 projection: the static scale of scaled_mm
        dict(name="norm_token", op="norm", T=1, H=1920, dtype="bf16", q="e4m3", dynamic=False, residual=True),
        # a ragged batch of mixed requests ahead of an int8 product; no size is a multiple of anything
        dict(name="norm_odd_int8", op="norm", T=777, H=1111, dtype="f16", q="int8", dynamic=True, residual=True),
        # a prompt of 8192 tokens at the projection's width, a scale for each token
        dict(name="norm_prefill", op="norm", T=8192, H=5760, dtype="bf16", q="e4m3", dynamic=True, residual=True),
        # fine-tuning on one short sequence
        dict(name="norm_grad_short", op="norm_grad", T=256, H=1920, dtype="bf16", residual=True),
        # a training step's batch of tokens at the projection's width
        dict(name="norm_grad_batch", op="norm_grad", T=8192, H=5760, dtype="bf16", residual=True),
        # one token through a projection (5760 x 1920): all of the time is in reading the weights
        dict(name="int8_token", op="int8", M=1, N=5760, K=1920, dtype="bf16"),
        # the linear layer of 64 tokens: a batch of decode steps
        dict(name="int8_linear", op="int8", M=64, N=5760, K=1920, dtype="bf16"),
        # the projection batch of 8192 tokens: bound by products
        dict(name="int8_projection", op="int8", M=8192, N=5760, K=1920, dtype="bf16"),
        # one sampled token's log probability with 20 alternatives from a large vocabulary
        dict(name="logprob_token", op="logprob", T=1, V=131072, dtype="f32", k=20, masked=0.0),
        # scoring a long batch against a large vocabulary, the logits as a bf16 head leaves them
        dict(name="logprob_score", op="logprob", T=4095, V=131072, dtype="bf16", k=5, masked=0.0),
        # training on a byte-like vocabulary: many rows, each of them short
        dict(name="logprob_grad_bytes", op="logprob_grad", T=8192, V=512, dtype="bf16", masked=0.0),
        # training with an entropy bonus on an odd vocabulary, some words never allowed
        dict(name="logprob_grad_vocab", op="logprob_grad", T=2047, V=50001, dtype="bf16", masked=0.1),
    ]


def _size(rng, low, high):
    """A whole number whose logarithm is spread evenly over [low, high]."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    n = max(low, min(high, n))
    return n - 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "int8", "logprob", "logprob_grad"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    es = _ES[dtype]
    if op in ("norm", "norm_grad"):
        H = _size(rng, 64, 8192)
        residual = rng.random() < 0.75
        case = dict(op=op, H=H, dtype=dtype, residual=residual)
        per = es * (3 if residual else 1) + 1 if op == "norm" else es * (4 if residual else 3)
        limit = _NORM_BYTES if op == "norm" else _GRAD_BYTES
        if op == "norm":
            case.update(q=rng.choice(["e4m3", "e5m2", "int8"]), dynamic=rng.random() < 0.6)
        case["T"] = _size(rng, 1, min(8192, int(limit * 0.99) // (H * per)))
        return case
    if op == "int8":
        N, K = _size(rng, 16, 8192), _size(rng, 16, 8192)
        M = _size(rng, 1, max(1, min(8192, _INT8_PRODUCTS // (N * K))))
        return dict(op=op, M=M, N=N, K=K, dtype=dtype)
    V = _size(rng, 64, 131072)
    masked = rng.choice([0.0, 0.0, 0.1, 0.9])
    case = dict(op=op, V=V, dtype=dtype, masked=masked)
    if op == "logprob":
        case["k"] = rng.choice([0, 1, 5, 20, 32])
        most = int(_LOGIT_BYTES * 0.99) // (V * es)
    else:
        most = int(_LOGIT_GRAD_BYTES * 0.99) // (2 * V * es)
    case["T"] = _size(rng, 1, min(8192, most))
    return case


def work(case):
    op = case["op"]
    if op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + M * N * _ES[case["dtype"]] + 4 * (M + N), "flops": 2 * M * N * K}
    es, T = _ES[case["dtype"]], case["T"]
    if op == "norm":
        H = case["H"]
        per_row = H * (es * (3 if case["residual"] else 1) + 1) + 4 + (4 if case["dynamic"] else 0)
        return {"bytes": T * per_row + H * es, "flops": 8 * T * H}
    if op == "norm_grad":
        H = case["H"]
        return {"bytes": T * (H * es * (4 if case["residual"] else 3) + 4) + H * (es + 4), "flops": 10 * T * H}
    V = case["V"]
    if op == "logprob":
        return {"bytes": T * (V * es + 8 + 24 + 12 * case["k"]), "flops": 6 * T * V}
    return {"bytes": T * (2 * V * es + 8 + 20), "flops": 8 * T * V}


# ---------------------------------------------------------------------------- inputs
def _logits(case, g, dev):
    """Logits of a trained head: near-normal, a few words far ahead of the others in each
    row; ``masked`` of the vocabulary at -inf, and one row of a masked batch wholly so."""
    T, V = case["T"], case["V"]
    x = torch.randn(T, V, generator=g, device=dev, dtype=torch.float32).mul_(2.5)
    lead = torch.randint(0, V, (T, 3), generator=g, device=dev)
    x.scatter_add_(1, lead, 8.0 * torch.rand(T, 3, generator=g, device=dev))
    if case["masked"] > 0:
        x.masked_fill_(torch.rand(V, generator=g, device=dev)[None, :] < case["masked"], -math.inf)
        if T >= 8:
            x[T // 2] = -math.inf
    tokens = torch.randint(0, V, (T,), generator=g, device=dev)
    tokens[torch.rand(T, generator=g, device=dev) < 0.05] = _IGNORE      # padding
    return x.to(_DT[case["dtype"]]), tokens


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    if op in ("norm", "norm_grad"):
        T, H, dt = case["T"], case["H"], _DT[case["dtype"]]
        # tokens of different sizes and a few large channels, as a residual stream has them
        rows = torch.exp(0.5 * randn(T, 1))
        cols = torch.where(torch.rand(H, generator=g, device=dev) < 0.01, 12.0, 1.0)
        s["weight"] = (1.0 + 0.2 * randn(H)).to(dt)
        if op == "norm":
            s["x"] = (randn(T, H) * 0.7).to(dt)
            if case["residual"]:
                s["residual"] = (randn(T, H) * rows * cols).to(dt)
            else:
                s["x"] = (randn(T, H) * rows * cols).to(dt)
            if not case["dynamic"]:      # calibrated: twelve standard deviations reach the largest code
                s["scale"] = torch.full((1,), 12.0 / _QMAX[case["q"]], device=dev)
        else:
            s["hidden"] = (randn(T, H) * rows * cols).to(dt)
            s["rstd"] = (s["hidden"].float().square().mean(-1) + _EPS).rsqrt()
            s["grad_y"] = (randn(T, H) * 0.05).to(dt)
            if case["residual"]:
                s["grad_residual"] = (randn(T, H) * 0.05).to(dt)
    elif op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"] = (randn(M, K) * 32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["w"] = (randn(N, K) * 32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["scale_a"] = 0.01 + 0.03 * torch.rand(M, generator=g, device=dev)
        s["scale_b"] = 0.001 + 0.002 * torch.rand(N, generator=g, device=dev)
    else:
        s["logits"], s["tokens"] = _logits(case, g, dev)
        if op == "logprob_grad":             # what the forward call left: each row's peak, log z and entropy
            peak = s["logits"].amax(-1).float()
            t = s["logits"].float() - peak.clamp_min(torch.finfo(torch.float32).min)[:, None]
            e = t.exp()
            z = e.sum(-1)
            entropy = torch.where(z > 0, z.log() - (e * t.clamp_min(-1e4)).sum(-1) / z, 0.0)
            s["stats"] = torch.stack([peak, z.log(), entropy], 1)
            s["grad_logprob"] = -torch.rand(case["T"], generator=g, device=dev)      # weights of a summed loss
            s["grad_entropy"] = 0.1 * randn(case["T"])
    return s


# ------------------------------------------------------------------------ plain forms
def _plain_norm(s):
    case = s["case"]
    h = s["x"].float()
    if case["residual"]:
        h = h + s["residual"].float()
    rstd = (h.square().mean(-1) + _EPS).rsqrt()
    y = h * rstd[:, None] * s["weight"].float()
    qmax = _QMAX[case["q"]]
    if case["dynamic"]:
        scale = (y.abs().amax(-1) / qmax).clamp_min(_SCALE_MIN)
        v = y / scale[:, None]
    else:
        scale = s["scale"]
        v = y / scale
    q = v.round().clamp(-128, 127).to(torch.int8) if case["q"] == "int8" else v.clamp(-qmax, qmax).to(_QT[case["q"]])
    return q, scale, h.to(s["x"].dtype), rstd


def _plain_norm_grad(s):
    w, h, gy, rstd = s["weight"].float(), s["hidden"].float(), s["grad_y"].float(), s["rstd"]
    g = gy * w
    c = (g * h).mean(-1) * rstd * rstd
    gx = rstd[:, None] * (g - h * c[:, None])
    if s["case"]["residual"]:
        gx = gx + s["grad_residual"].float()
    return gx.to(s["hidden"].dtype), (gy * h * rstd[:, None]).sum(0)


def _plain_int8(s):
    acc = s["a"].float() @ s["w"].float().t()
    return (acc * s["scale_a"][:, None] * s["scale_b"]).to(_DT[s["case"]["dtype"]])


def _plain_logprob(s):
    k = s["case"]["k"]
    x = s["logits"].float()
    V = x.shape[1]
    m = x.amax(-1).clamp_min(torch.finfo(torch.float32).min)
    t = x - m[:, None]
    e = t.exp()
    z = e.sum(-1)
    some = z > 0
    logz = z.log()
    entropy = torch.where(some, logz - (e * t.clamp_min(-1e4)).sum(-1) / z, 0.0)
    del e
    keep = s["tokens"] != _IGNORE
    at = t.gather(1, torch.where(keep, s["tokens"], 0)[:, None])[:, 0]
    logprob = torch.where(keep, torch.where(some, at - logz, -math.inf), 0.0)
    stats = torch.stack([x.amax(-1), logz, entropy], 1)
    # one 64-bit key for each logit: its order among floats above, the lower index first below
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64)
    key = order * (1 << 32) + ((1 << 31) - 1 - torch.arange(V, device=x.device))
    top = key.topk(k, dim=-1).values
    ids = (1 << 31) - 1 - (top & 0xFFFFFFFF)
    lead = torch.where(some[:, None], t.gather(1, ids) - logz[:, None], -math.inf)
    return logprob, entropy, torch.where(some, m + logz, -math.inf), stats, lead, ids


def _plain_logprob_grad(s):
    x = s["logits"].float()
    V = x.shape[1]
    peak, logz, entropy = (c[:, None] for c in s["stats"].unbind(1))
    some = peak > -math.inf
    lp = torch.where(some, x - peak - logz, -math.inf)
    p = lp.exp()
    g = torch.where(s["tokens"] != _IGNORE, s["grad_logprob"], 0.0)[:, None]
    hot = (torch.arange(V, device=x.device) == s["tokens"][:, None]) & some
    out = g * (hot.float() - p) - s["grad_entropy"][:, None] * p * (lp.clamp_min(-1e4) + entropy)
    return out.to(s["logits"].dtype)


# ------------------------------------------------------------------------------- runs
def _norm_outputs(case, q, scale, residual, rstd):
    if case["q"] == "int8":              # int8 codes as the values that they stand for
        held = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        q = torch.mul(q, scale[:, None] if case["dynamic"] else scale, out=held)
    out = {"q": q, "rstd": rstd}
    if case["residual"]:
        out["residual"] = residual
    if case["dynamic"]:
        out["scale"] = scale
    return out


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        if op == "norm":
            return _norm_outputs(case, *_plain_norm(s))
        if op == "norm_grad":
            gx, gw = _plain_norm_grad(s)
            return {"grad_x": gx, "grad_weight": gw}
        if op == "int8":
            return {"out": _plain_int8(s)}
        if op == "logprob":
            logprob, entropy, lse, stats, lead, ids = _plain_logprob(s)
        else:
            return {"grad_logits": _plain_logprob_grad(s)}
    else:
        import bit_exact_fp8_gb300 as fw
        if op == "norm":
            r = fw.rms_norm_quant(s["x"], s["weight"], s.get("residual"), eps=_EPS, out_dtype=_QT[case["q"]],
                                  scale=s.get("scale"))
            return _norm_outputs(case, r.q, r.scale, r.residual, r.rstd)
        if op == "norm_grad":
            gx, gw = fw.rms_norm_backward(s["grad_y"], s["hidden"], s["rstd"], s["weight"], s.get("grad_residual"))
            return {"grad_x": gx, "grad_weight": gw}
        if op == "int8":
            return {"out": fw.int8_scaled_mm(s["a"], s["w"].t(), s["scale_a"], s["scale_b"],
                                             out_dtype=_DT[case["dtype"]])}
        if op == "logprob":
            logprob, entropy, lse, stats, lead, ids = fw.token_logprobs(s["logits"], s["tokens"], top_k=case["k"],
                                                                        ignore_index=_IGNORE)
        else:
            return {"grad_logits": fw.token_logprobs_backward(s["logits"], s["tokens"], s["stats"],
                                                              s["grad_logprob"], s["grad_entropy"],
                                                              ignore_index=_IGNORE)}
    out = {"logprob": logprob, "entropy": entropy, "lse": lse, "stats": stats}
    if case["k"] > 0:
        out["top_logprobs"], out["top_ids"] = lead, ids
    return out


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "norm":
        h = s["x"].to(f64)
        if case["residual"]:
            h += s["residual"].to(f64)
        rstd = 1.0 / torch.sqrt(torch.sum(h * h, dim=1) / case["H"] + _EPS)
        y = h * s["weight"].to(f64) * rstd.unsqueeze(1)
        top = _QMAX[case["q"]]
        if case["dynamic"]:
            scale = torch.clamp(torch.max(y.abs(), dim=1).values / top, min=_SCALE_MIN)
        else:
            scale = s["scale"].to(f64)
        y = y / (scale.unsqueeze(1) if case["dynamic"] else scale)
        if case["q"] == "int8":
            q = torch.clamp(torch.round(y), -128, 127)
            q = q * (scale.unsqueeze(1) if case["dynamic"] else scale)
        else:                            # to the nearest code, ties to even, none above the largest
            bits, low = (3, -6) if case["q"] == "e4m3" else (2, -14)
            e = torch.clamp(torch.frexp(y)[1].to(f64) - 1, min=low)
            step = torch.exp2(e - bits)
            q = torch.clamp(torch.round(y / step) * step, -top, top)
        out = {"q": q, "rstd": rstd}
        if case["residual"]:
            out["residual"] = h
        if case["dynamic"]:
            out["scale"] = scale
        return out
    if op == "norm_grad":
        gy, h, w, r = s["grad_y"].to(f64), s["hidden"].to(f64), s["weight"].to(f64), s["rstd"].to(f64)
        n = h * r.unsqueeze(1)           # the normalised rows
        gn = gy * w
        gx = r.unsqueeze(1) * (gn - n * (torch.sum(gn * n, dim=1) / case["H"]).unsqueeze(1))
        if case["residual"]:
            gx += s["grad_residual"].to(f64)
        return {"grad_x": gx, "grad_weight": torch.einsum("th,th->h", gy, n)}
    if op == "int8":
        acc = torch.mm(s["a"].to(f64), s["w"].to(f64).t())
        return {"out": torch.einsum("mn,m,n->mn", acc, s["scale_a"].to(f64), s["scale_b"].to(f64))}
    x = s["logits"].to(f64)
    empty = torch.isneginf(x).all(dim=1)
    if op == "logprob":
        lse = torch.logsumexp(x, dim=1)
        p = torch.softmax(x, dim=1)
        entropy = torch.special.entr(p).sum(dim=1).masked_fill(empty, 0.0)
        del p
        pad = s["tokens"] == _IGNORE
        at = x[torch.arange(case["T"], device=x.device), s["tokens"].masked_fill(pad, 0)]
        logprob = (at - lse).masked_fill(empty, -math.inf).masked_fill(pad, 0.0)
        peak = torch.max(x, dim=1).values
        out = {"logprob": logprob, "entropy": entropy, "lse": lse,
               "stats": torch.stack([peak, (lse - peak).masked_fill(empty, -math.inf), entropy], dim=1)}
        if case["k"] > 0:
            lead = torch.topk(x, case["k"], dim=1).values - lse.unsqueeze(1)
            out["top_logprobs"] = lead.masked_fill(empty.unsqueeze(1), -math.inf)
            out["top_ids"] = None
        return out
    # d logprob / d x_v = [v = token] - p_v;  d entropy / d x_v = -p_v (log p_v + entropy)
    peak, logz, entropy = s["stats"].to(f64).unsqueeze(2).unbind(1)
    p = torch.exp(x - peak - logz)
    pad = s["tokens"] == _IGNORE
    gl = s["grad_logprob"].to(f64).masked_fill(pad, 0.0)
    part = torch.special.entr(p) - p * entropy
    gx = part * s["grad_entropy"].to(f64).unsqueeze(1) - gl.unsqueeze(1) * p
    rows = torch.arange(case["T"], device=x.device)
    gx[rows, s["tokens"].masked_fill(pad, 0)] += gl
    return {"grad_logits": gx.masked_fill(empty.unsqueeze(1), 0.0)}

"""The operators of 8-bit layers with block scales, as cases to be measured: quantisation in
blocks of 128, the FP8 product with a scale for each block, the same product by expert over
ragged groups of rows with its weights' gradient, and SwiGLU with its inputs kept in 8 bits
for the backward pass.

A case is a dict of plain values; ``op`` names the operator.  ``run`` computes it by
elementary torch operations in 32 bits, or, with ``own`` true, through this package.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_ES = {"bf16": 2, "f16": 2, "f32": 4}
_QT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_QMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_SCALE_MIN = 2.0 ** -126
# what shares a scale: 128 values of a row, 128 of a column, or a square of both
_BLOCK = {"rows": (1, 128), "columns": (128, 1), "squares": (128, 128)}

# the most that one drawn case may need
_QUANT_BYTES = 8192 * 5760 * 3
_SWIGLU_BYTES = 8192 * 5760 * 7
_SWIGLU_GRAD_BYTES = 8192 * 5760 * 8
_MM_PRODUCTS = 8192 * 5760 * 1920
_GROUPED_PRODUCTS = 8191 * 5760 * 1920
_GROUPED_WEIGHTS = 32 * 5760 * 1920


def listed():
    return [
        # one new token's activations ahead of a decode step's projection
        dict(name="quant_token", op="quant", T=1, H=1920, dtype="bf16", q="e4m3", block="rows"),
        # a training batch's activations, kept in 8 bits: the forward product and the weights' gradient read the same codes
        dict(name="quant_batch", op="quant", T=8192, H=5760, dtype="bf16", q="e4m3", block="squares"),
        # one token through a projection: all of the time is in reading the weights
        dict(name="mm_token", op="mm", layout="forward", M=1, N=5760, K=1920, fa="e4m3", fb="e4m3", block="rows", dtype="bf16"),
        # the linear layer of 64 tokens: a batch of decode steps
        dict(name="mm_linear", op="mm", layout="forward", M=64, N=5760, K=1920, fa="e4m3", fb="e4m3", block="rows", dtype="bf16"),
        # the projection batch of 8192 tokens: bound by products
        dict(name="mm_projection", op="mm", layout="forward", M=8192, N=5760, K=1920, fa="e4m3", fb="e4m3", block="rows",
             dtype="bf16"),
        # the gradient of an odd number of tokens by the layer's input: the weights are read across their rows
        dict(name="mm_input_grad", op="mm", layout="input_grad", M=777, N=1920, K=5760, fa="e5m2", fb="e4m3", block="rows",
             dtype="bf16"),
        # the gradient by the weights, both operands read across their rows, with a scale for each column
        dict(name="mm_weight_grad", op="mm", layout="weight_grad", M=5760, N=1920, K=8192, fa="e5m2", fb="e4m3",
             block="columns", dtype="f32"),
        # a decode step of 16 tokens that take 8 experts each: most experts have a row or two, some none
        dict(name="grouped_decode", op="grouped", layout="forward", T=128, E=64, N=1920, K=1920, fa="e4m3", fb="e4m3",
             tail=False, dtype="bf16"),
        # a ragged prompt batch over experts of unequal favour, with rows of padding behind the last group
        dict(name="grouped_prompt", op="grouped", layout="forward", T=8191, E=32, N=5760, K=1920, fa="e4m3", fb="e4m3",
             tail=True, dtype="bf16"),
        # the experts' weights' gradients in a training step
        dict(name="grouped_weight_grad", op="grouped_grad", T=4099, E=8, N=1920, K=1920, fa="e5m2", fb="e4m3",
             block="squares", tail=False, dtype="f32"),
        # a small batch of requests through the middle of an MLP; no size is a multiple of anything
        dict(name="swiglu_odd", op="swiglu", T=77, H=1111, dtype="f16", q="e4m3", block="rows"),
        # the backward pass of a training batch from the 8-bit checkpoint
        dict(name="swiglu_grad_batch", op="swiglu_grad", T=8192, H=5760, dtype="bf16"),
    ]


def _size(rng, low, high, step=1):
    """A multiple of `step` (or a bound) whose logarithm is spread evenly over [low, high]."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    n = -(-n // step) * step
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["quant", "mm", "mm", "grouped", "grouped", "grouped_grad", "swiglu", "swiglu_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    es = _ES[dtype]
    step = rng.choice([128, 16, 16, 1])          # most models' widths are multiples of something
    if op in ("quant", "swiglu", "swiglu_grad"):
        H = _size(rng, 64, 8192, step)
        case = dict(op=op, H=H, dtype=dtype)
        if op == "quant":
            per, limit = es + 1, _QUANT_BYTES
            case.update(q=rng.choice(["e4m3", "e5m2"]), block=rng.choice(["rows", "columns", "squares"]))
        elif op == "swiglu":
            per, limit = 2 * es + 3, _SWIGLU_BYTES
            case.update(q=rng.choice(["e4m3", "e5m2"]), block=rng.choice(["rows", "squares"]))
        else:
            per, limit = 3 * es + 2, _SWIGLU_GRAD_BYTES
        case["T"] = _size(rng, 1, min(8192, int(limit * 0.99) // (H * per)))
        return case
    fa, fb = rng.choice([("e4m3", "e4m3"), ("e4m3", "e4m3"), ("e5m2", "e4m3")])
    if op == "mm":
        layout = rng.choice(["forward", "forward", "input_grad", "weight_grad"])
        N, K = _size(rng, 16, 8192, step), _size(rng, 16, 8192, step)
        M = _size(rng, 1, max(1, min(8192, _MM_PRODUCTS // (N * K))), step if layout == "weight_grad" else 1)
        block = rng.choice(["columns", "squares"] if layout == "weight_grad" else ["rows", "rows", "squares"])
        return dict(op=op, layout=layout, M=M, N=N, K=K, fa=fa, fb=fb, block=block, dtype=dtype)
    N, K = _size(rng, 64, 4096, step), _size(rng, 64, 4096, step)
    E = _size(rng, 1, max(1, min(128, _GROUPED_WEIGHTS // (N * K * (4 if op == "grouped_grad" else 1)))))
    T = _size(rng, 1, max(1, min(8191, _GROUPED_PRODUCTS // (N * K))))
    case = dict(op=op, T=T, E=E, N=N, K=K, fa=fa, fb=fb, tail=rng.random() < 0.3, dtype=dtype)
    if op == "grouped":
        case["layout"] = rng.choice(["forward", "forward", "input_grad"])
    else:
        case["block"] = rng.choice(["columns", "squares"])
    return case


def _blocks(n):
    return -(-n // 128)


def _scales(rows, cols, block):
    br, bc = _BLOCK[block]
    return -(-rows // br) * -(-cols // bc)


def work(case):
    op = case["op"]
    if op in ("quant", "swiglu", "swiglu_grad"):
        T, H, es = case["T"], case["H"], _ES[case["dtype"]]
        if op == "quant":
            return {"bytes": T * H * (es + 1) + 4 * _scales(T, H, case["block"]), "flops": 4 * T * H}
        kept = 2 * T * H + 8 * T * _blocks(H)
        if op == "swiglu":
            return {"bytes": T * H * (2 * es + 1) + kept + 4 * _scales(T, H, case["block"]), "flops": 20 * T * H}
        return {"bytes": 3 * T * H * es + kept, "flops": 20 * T * H}
    es, N, K = _ES[case["dtype"]], case["N"], case["K"]
    if op == "mm":
        M = case["M"]
        if case["layout"] == "weight_grad":
            scales = _scales(K, M, case["block"]) + _scales(K, N, case["block"])
        else:
            scales = _scales(M, K, case["block"]) + _blocks(N) * _blocks(K)
        return {"bytes": M * K + N * K + M * N * es + 4 * scales, "flops": 2 * M * N * K}
    T, E = case["T"], case["E"]
    if op == "grouped":
        rows, used = T * (0.9 if case["tail"] else 1.0), min(E, T)
        return {"bytes": int(rows * K) + T * N * es + used * (N * K + 4 * _blocks(N) * _blocks(K)) + 4 * T * _blocks(K),
                "flops": int(2 * rows * N * K)}
    scales = _scales(T, N, case["block"]) + _scales(T, K, case["block"])
    return {"bytes": T * (N + K) + E * N * K * es + 4 * scales, "flops": 2 * T * N * K}


# ---------------------------------------------------------------------------- inputs
def _per_value(scale, block, shape):
    """The scale of each value of the last two dimensions, as a view of their size."""
    br, bc = _BLOCK[block]
    if br > 1:
        scale = scale.repeat_interleave(br, -2)[..., :shape[-2], :]
    if bc > 1:
        scale = scale.repeat_interleave(bc, -1)[..., :shape[-1]]
    return scale


def _quantise(x, block, fmt):
    """(codes, scales) of the last two dimensions of x, by elementary operations in 32 bits."""
    br, bc = _BLOCK[block]
    rows, cols = x.shape[-2:]
    y = x.float()
    a = torch.nn.functional.pad(y.abs(), (0, -cols % bc, 0, -rows % br))
    a = a.unflatten(-1, (-1, bc)).unflatten(-3, (-1, br)).amax((-1, -3))
    scale = (a / _QMAX[fmt]).clamp_min(_SCALE_MIN)
    v = y / _per_value(scale, block, y.shape)
    return v.clamp(-_QMAX[fmt], _QMAX[fmt]).to(_QT[fmt]), scale


def _value(codes, scale, block):
    return codes.float() * _per_value(scale, block, codes.shape)


def _groups(case, seed):
    """Rows for each expert: unequal favour, some with none; with `tail`, a tenth of the rows behind the last."""
    T, E = case["T"], case["E"]
    rng = random.Random(seed * 1000003 + T * 131 + E)
    rows = T - T // 10 if case["tail"] else T
    favour = [0.0 if rng.random() < 0.1 else rng.gammavariate(2.0, 1.0) for _ in range(E)]
    if not any(favour):
        favour[rng.randrange(E)] = 1.0
    total, reached, ends, cut = sum(favour), 0.0, [0], 0
    for f in favour:
        reached += f
        cut = max(cut, min(rows, int(round(rows * reached / total))))
        ends.append(cut)
    ends[-1] = rows
    return ends


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def acts(rows, cols):
        """Activations of a residual stream: tokens of different sizes, a few large channels."""
        size = torch.exp(0.5 * randn(rows, 1))
        large = torch.where(torch.rand(cols, generator=g, device=dev) < 0.01, 12.0, 1.0)
        return randn(rows, cols).mul_(size).mul_(large)

    if op == "quant":
        s["x"] = acts(case["T"], case["H"]).to(_DT[case["dtype"]])
        return s
    if op == "swiglu":
        s["gate_up"] = acts(case["T"], 2 * case["H"]).to(_DT[case["dtype"]])
        return s
    if op == "swiglu_grad":
        T, H = case["T"], case["H"]
        gu = acts(T, 2 * H)
        s["checkpoint"], s["checkpoint_scale"] = _quantise_halves(gu.to(_DT[case["dtype"]]), "e4m3")
        s["grad_y"] = (randn(T, H) * 0.05).to(_DT[case["dtype"]])
        return s
    N, K, fa, fb = case["N"], case["K"], case["fa"], case["fb"]
    if op == "mm":
        M = case["M"]
        if case["layout"] == "weight_grad":               # of K tokens: gradients [K, M] and activations [K, N]
            s["a"], s["scale_a"] = _quantise(randn(K, M).mul_(0.05), case["block"], fa)
            s["b"], s["scale_b"] = _quantise(acts(K, N), case["block"], fb)
        else:
            s["a"], s["scale_a"] = _quantise(acts(M, K), case["block"], fa)
            shape = (N, K) if case["layout"] == "forward" else (K, N)
            s["b"], s["scale_b"] = _quantise(randn(*shape).mul_(K ** -0.5), "squares", fb)
        return s
    s["ends"] = _groups(case, seed)                       # a plain program walks the groups on the host
    s["offsets"] = torch.tensor(s["ends"], dtype=torch.int32, device=dev)
    T, E = case["T"], case["E"]
    if op == "grouped":
        s["a"], s["scale_a"] = _quantise(acts(T, K), "rows", fa)
        shape = (N, K) if case["layout"] == "forward" else (K, N)
        s["b"] = torch.empty(E, *shape, dtype=_QT[fb], device=dev)
        s["scale_b"] = torch.empty(E, *(_blocks(n) for n in shape), device=dev)
        for e in range(E):
            s["b"][e], s["scale_b"][e] = _quantise(randn(*shape).mul_(K ** -0.5), "squares", fb)
    else:
        s["a"], s["scale_a"] = _quantise(randn(T, N).mul_(0.05), case["block"], fa)
        s["b"], s["scale_b"] = _quantise(acts(T, K), case["block"], fb)
    return s


# ------------------------------------------------------------------------ plain forms
def _quantise_halves(x, fmt):
    """The gate's half and the other in blocks of their own."""
    parts = [_quantise(h, "rows", fmt) for h in x.chunk(2, -1)]
    codes = torch.cat([p[0].view(torch.uint8) for p in parts], -1).view(_QT[fmt])
    return codes, torch.cat([p[1] for p in parts], -1)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quant":
        q, scale = _quantise(s["x"], case["block"], case["q"])
        return {"q": q, "scale": scale}
    if op == "swiglu":
        gate, up = s["gate_up"].float().chunk(2, -1)
        y = gate * up / (1.0 + torch.exp(-gate))
        q, scale = _quantise(y, case["block"], case["q"])
        kept, kept_scale = _quantise_halves(s["gate_up"], "e4m3")
        return {"q": q, "scale": scale, "checkpoint": kept, "checkpoint_scale": kept_scale}
    if op == "swiglu_grad":
        scales = s["checkpoint_scale"].chunk(2, -1)
        gate, up = (_value(s["checkpoint"][:, h], k, "rows") for h, k in zip(_halves(case["H"]), scales))
        gy = s["grad_y"].float()
        sig = 1.0 / (1.0 + torch.exp(-gate))
        grad_gate = gy * up * sig * (1.0 + gate * (1.0 - sig))
        return {"grad_gate_up": torch.cat([grad_gate, gy * gate * sig], -1).to(s["grad_y"].dtype)}
    dt = _DT[case["dtype"]]
    if op == "mm":
        if case["layout"] == "weight_grad":
            a, b = _value(s["a"], s["scale_a"], case["block"]), _value(s["b"], s["scale_b"], case["block"])
            return {"out": (a.t() @ b).to(dt)}
        a, b = _value(s["a"], s["scale_a"], case["block"]), _value(s["b"], s["scale_b"], "squares")
        return {"out": (a @ (b.t() if case["layout"] == "forward" else b)).to(dt)}
    ends = s["ends"]
    if op == "grouped":
        out = torch.zeros(case["T"], case["N"], dtype=dt, device=s["a"].device)
        a = _value(s["a"], s["scale_a"], "rows")
        for e in range(case["E"]):
            if ends[e + 1] > ends[e]:
                w = _value(s["b"][e], s["scale_b"][e], "squares")
                out[ends[e]:ends[e + 1]] = (a[ends[e]:ends[e + 1]] @ (w.t() if case["layout"] == "forward" else w)).to(dt)
        return {"out": out}
    a, b = _value(s["a"], s["scale_a"], case["block"]), _value(s["b"], s["scale_b"], case["block"])
    out = torch.empty(case["E"], case["N"], case["K"], dtype=dt, device=a.device)
    for e in range(case["E"]):
        out[e] = (a[ends[e]:ends[e + 1]].t() @ b[ends[e]:ends[e + 1]]).to(dt)
    return {"out": out}


def _halves(H):
    return slice(0, H), slice(H, 2 * H)


# ------------------------------------------------------------------------------- runs
def run(state):
    s, case = state, state["case"]
    if not own:
        return _plain(s)
    import bit_exact_fp8_gb300 as fw
    op = case["op"]
    if op == "quant":
        q, scale = fw.block_quant(s["x"], block=_BLOCK[case["block"]], out_dtype=_QT[case["q"]])
        return {"q": q, "scale": scale}
    if op == "swiglu":
        r = fw.swiglu_quant(s["gate_up"], block=_BLOCK[case["block"]], out_dtype=_QT[case["q"]], checkpoint=True)
        return {"q": r.q, "scale": r.scale, "checkpoint": r.checkpoint, "checkpoint_scale": r.checkpoint_scale}
    if op == "swiglu_grad":
        return {"grad_gate_up": fw.swiglu_backward(s["grad_y"], s["checkpoint"], s["checkpoint_scale"])}
    dt = _DT[case["dtype"]]
    if op == "mm":
        if case["layout"] == "weight_grad":
            return {"out": fw.block_scaled_mm(s["a"].t(), s["b"], s["scale_a"].t(), s["scale_b"], out_dtype=dt)}
        b, scale_b = s["b"], s["scale_b"]
        if case["layout"] == "forward":
            b, scale_b = b.t(), scale_b.t()
        return {"out": fw.block_scaled_mm(s["a"], b, s["scale_a"], scale_b, out_dtype=dt)}
    if op == "grouped":
        b, scale_b = s["b"], s["scale_b"]
        if case["layout"] == "forward":
            b, scale_b = b.transpose(1, 2), scale_b.transpose(1, 2)
        return {"out": fw.grouped_block_scaled_mm(s["a"], b, s["offsets"], s["scale_a"], scale_b, out_dtype=dt)}
    return {"out": fw.grouped_block_scaled_wgrad(s["a"], s["b"], s["offsets"], s["scale_a"], s["scale_b"], out_dtype=dt)}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_quant(x, block, fmt):
    """(codes' values, scales): each value over its block's scale, to the nearest code, ties to even."""
    br, bc = _BLOCK[block]
    rows, cols = x.shape
    top = _QMAX[fmt]
    held = torch.zeros(_scales(rows, 1, "columns") * 128, _blocks(cols) * 128, dtype=torch.float64, device=x.device)
    held[:rows, :cols] = x.abs()
    if bc > 1:
        held = held.reshape(held.shape[0], -1, bc).max(2).values
    if br > 1:
        held = held.reshape(-1, br, held.shape[1]).max(1).values
    scale = (held / top).clamp(min=_SCALE_MIN)[:-(-rows // br), :-(-cols // bc)]
    r, c = torch.arange(rows, device=x.device) // br, torch.arange(cols, device=x.device) // bc
    v = x / scale[r][:, c]
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    step = torch.exp2((torch.frexp(v)[1].to(torch.float64) - 1).clamp(min=low) - bits)
    return torch.clamp(torch.round(v / step) * step, -top, top), scale


def _exact_value(codes, scale, block):
    br, bc = _BLOCK[block]
    r, c = torch.arange(codes.shape[0], device=codes.device) // br, torch.arange(codes.shape[1], device=codes.device) // bc
    return codes.to(torch.float64) * scale.to(torch.float64)[r][:, c]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "quant":
        q, scale = _exact_quant(s["x"].to(f64), case["block"], case["q"])
        return {"q": q, "scale": scale}
    if op in ("swiglu", "swiglu_grad"):
        H = case["H"]
        left, right = _halves(H)
        if op == "swiglu":
            x = s["gate_up"].to(f64)
            q, scale = _exact_quant(torch.sigmoid(x[:, left]) * x[:, left] * x[:, right], case["block"], case["q"])
            kept = [_exact_quant(x[:, h], "rows", "e4m3") for h in (left, right)]
            return {"q": q, "scale": scale, "checkpoint": torch.cat([k[0] for k in kept], 1),
                    "checkpoint_scale": torch.cat([k[1] for k in kept], 1)}
        n = _blocks(H)
        gate = _exact_value(s["checkpoint"][:, left], s["checkpoint_scale"][:, :n], "rows")
        up = _exact_value(s["checkpoint"][:, right], s["checkpoint_scale"][:, n:], "rows")
        gy, sig = s["grad_y"].to(f64), torch.sigmoid(gate)
        return {"grad_gate_up": torch.cat([gy * up * (sig + gate * sig * torch.sigmoid(-gate)), gy * gate * sig], 1)}
    if op == "mm":
        a_block = case["block"]
        a = _exact_value(s["a"], s["scale_a"], a_block)
        if case["layout"] == "weight_grad":
            return {"out": torch.einsum("km,kn->mn", a, _exact_value(s["b"], s["scale_b"], a_block))}
        b = _exact_value(s["b"], s["scale_b"], "squares")
        return {"out": torch.einsum("mk,nk->mn" if case["layout"] == "forward" else "mk,kn->mn", a, b)}
    ends = s["ends"]
    if op == "grouped":
        out = torch.zeros(case["T"], case["N"], dtype=f64, device=s["a"].device)
        for e in range(case["E"]):
            lo, hi = ends[e], ends[e + 1]
            if lo < hi:
                a = _exact_value(s["a"][lo:hi], s["scale_a"][lo:hi], "rows")
                b = _exact_value(s["b"][e], s["scale_b"][e], "squares")
                out[lo:hi] = torch.einsum("tk,nk->tn" if case["layout"] == "forward" else "tk,kn->tn", a, b)
        return {"out": out}
    a = _exact_value(s["a"], s["scale_a"], case["block"])
    b = _exact_value(s["b"], s["scale_b"], case["block"])
    parts = [torch.einsum("tn,tk->nk", a[lo:hi], b[lo:hi]) for lo, hi in zip(ends, ends[1:])]
    return {"out": torch.stack(parts)}

"""The sublayer operators between two mHC boundaries, in their plain form and as the framework's calls.

Operators (8-bit tensors are E4M3 values with one FP32 scale for each block of 128 along the row):

* norm      r = x + residual, y = r * rsqrt(mean(r^2) + eps) * weight; outputs r, y and y in 8 bits.
* quantize  x in 8 bits.
* swiglu    silu(gate) * up in 8 bits, gate and up the halves of each row.
* matmul    (a * a_scales) @ (w * w_scales)^T, w with one scale for each 128 x 128 block.
* moe       a whole mixture-of-experts layer: router, top-k, the chosen experts' gate, up and down
            products, the weighted sum, and the shared experts.

`own` chooses the form: False runs elementary torch operations in 32 bits, True the package's Sublayer.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100     # an all-zero block gets this maximum, so that no scale is zero
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the norm before a single token's projections, where only latency counts
        {"name": "norm_1", "op": "norm", "m": 1, "h": 5120},
        # the same in a prompt of 4096 tokens: the memory rate
        {"name": "norm_4096", "op": "norm", "m": 4096, "h": 6144},
        # a boundary's layer input of a decode batch, made ready for the 8-bit products
        {"name": "quantize_64", "op": "quantize", "m": 64, "h": 5120},
        # a ragged prompt with a width that ends inside a block of 128
        {"name": "quantize_1999", "op": "quantize", "m": 1999, "h": 5064},
        # the activation of a dense MLP for a few tokens, width not a multiple of 128
        {"name": "swiglu_7", "op": "swiglu", "m": 7, "h": 1944},
        # the same for a prompt
        {"name": "swiglu_4096", "op": "swiglu", "m": 4096, "h": 2048},
        # an attention output projection for one token: the weight's read is the time
        {"name": "matmul_1", "op": "matmul", "m": 1, "n": 6144, "k": 5120, "out": "bf16"},
        # a latent projection for a small odd batch, width not a multiple of 128, FP32 output
        {"name": "matmul_37", "op": "matmul", "m": 37, "n": 2120, "k": 5120, "out": "f32"},
        # gate and up of a dense MLP for a prompt: the tensor rate
        {"name": "matmul_4096", "op": "matmul", "m": 4096, "n": 4096, "k": 6144, "out": "bf16"},
        # one decoded token through a large layer with 8-bit weights and a shared expert
        {"name": "moe_1", "op": "moe", "m": 1, "h": 5120, "i": 2048, "experts": 64, "shared": 1, "top_k": 8,
         "fp8": True, "score": "softmax"},
        # five tokens through a small layer with BF16 weights, sigmoid scores and a selection bias
        {"name": "moe_5", "op": "moe", "m": 5, "h": 1024, "i": 512, "experts": 16, "shared": 0, "top_k": 2,
         "fp8": False, "score": "sigmoid"},
        # a decode batch of 32 that reaches nearly every expert
        {"name": "moe_32", "op": "moe", "m": 32, "h": 5120, "i": 2048, "experts": 64, "shared": 1, "top_k": 8,
         "fp8": True, "score": "softmax"},
    ]


def _log(rng, lo, hi, step=1):
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi and v != 3072:
            return v


def draw(rng):
    op = rng.choice(["norm", "quantize", "swiglu", "matmul", "matmul", "moe", "moe"])
    if op in ("norm", "quantize"):
        return {"op": op, "m": _log(rng, 1, 4096), "h": _log(rng, 128, 6144, 8)}
    if op == "swiglu":
        return {"op": op, "m": _log(rng, 1, 4096), "h": _log(rng, 64, 2048, 8)}
    if op == "matmul":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 64, 4096, 8), "k": _log(rng, 128, 6144, 16),
                "out": rng.choice(["bf16", "bf16", "f32"])}
    fp8 = rng.random() < 0.6
    experts = rng.randint(8, 64 if fp8 else 32)
    return {"op": op, "m": _log(rng, 1, 32), "h": _log(rng, 256, 5120, 16), "i": _log(rng, 128, 2048, 16),
            "experts": experts, "shared": rng.randint(0, 1), "top_k": rng.randint(1, min(8, experts)), "fp8": fp8,
            "score": rng.choice(["softmax", "sigmoid"])}


# ------------------------------------------------------------------ inputs
def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, m, h):
    """Rows as they leave a norm: unit scale, a few channels that are much larger."""
    gain = 1.0 + 12.0 * (torch.rand(h, generator=g, device="cuda") < 0.004)
    return _randn(g, m, h) * gain


def _fp8_values(g, *shape):
    return (_randn(g, *shape) * 110.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _fp8_scales(g, k, *shape):
    return (0.5 + torch.rand(*shape, generator=g, device="cuda")) / (110.0 * math.sqrt(k))


def prepare(case, seed):
    g, op, m = _gen(seed), case["op"], case["m"]
    s = {"case": case}
    f8 = dict(dtype=torch.float8_e4m3fn, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    if op in ("norm", "quantize", "swiglu"):
        h = case["h"]
        if op == "norm":
            s["inputs"] = {"x": (0.3 * _activations(g, m, h)).bfloat16(), "residual": (2.0 * _randn(g, m, h)).bfloat16(),
                           "norm_weight": (1.0 + 0.1 * _randn(g, h)).bfloat16()}
            s["outputs"] = {"residual_out": torch.empty(m, h, **bf16), "output": torch.empty(m, h, **bf16)}
        elif op == "quantize":
            s["inputs"] = {"x": _activations(g, m, h).bfloat16()}
            s["outputs"] = {}
        else:
            s["inputs"] = {"gate_up": (1.5 * _randn(g, m, 2 * h)).bfloat16()}
            s["outputs"] = {}
        s["outputs"]["values"] = torch.empty(m, h, **f8)
        s["outputs"]["scales"] = torch.empty(m, _blocks(h), **f32)
    elif op == "matmul":
        n, k = case["n"], case["k"]
        a = _activations(g, m, _blocks(k) * BLOCK).view(m, _blocks(k), BLOCK)
        scales = a.abs().amax(2) / E4M3_MAX
        values = (a / scales[:, :, None]).to(torch.float8_e4m3fn).view(m, -1)[:, :k].contiguous()
        s["inputs"] = {"values": values, "scales": scales, "weight": _fp8_values(g, n, k),
                       "weight_scales": _fp8_scales(g, k, _blocks(n), _blocks(k))}
        s["outputs"] = {"output": torch.empty(m, n, **(bf16 if case["out"] == "bf16" else f32))}
    else:
        h, i, e, sh = case["h"], case["i"], case["experts"], case["shared"]
        inputs = {"x": _activations(g, m, h).bfloat16(), "router": (_randn(g, e, h) / math.sqrt(h)).bfloat16()}
        if case["score"] == "sigmoid":
            inputs["bias"] = 0.05 * _randn(g, e)
        if case["fp8"]:
            inputs["gate_up"] = torch.empty(e + sh, 2 * i, h, **f8)
            inputs["down"] = torch.empty(e + sh, h, i, **f8)
            for j in range(e + sh):
                inputs["gate_up"][j] = _fp8_values(g, 2 * i, h)
                inputs["down"][j] = _fp8_values(g, h, i)
            inputs["gate_up_scales"] = _fp8_scales(g, h, e + sh, 2, _blocks(i), _blocks(h))
            inputs["down_scales"] = _fp8_scales(g, i, e + sh, _blocks(h), _blocks(i))
        else:
            inputs["gate_up"] = torch.empty(e + sh, 2 * i, h, **bf16)
            inputs["down"] = torch.empty(e + sh, h, i, **bf16)
            for j in range(e + sh):
                inputs["gate_up"][j] = _randn(g, 2 * i, h) / math.sqrt(h)
                inputs["down"][j] = _randn(g, h, i) / math.sqrt(i)
        s["inputs"] = inputs
        s["outputs"] = {"output": torch.empty(m, h, **bf16),
                        "idx": torch.empty(m, case["top_k"], dtype=torch.int32, device="cuda"),
                        "weights": torch.empty(m, case["top_k"], **f32)}
    if own:
        from mhc_residual_boundary_gb300 import Sublayer
        if op == "moe":
            s["sublayer"] = Sublayer(hidden=case["h"], intermediate=case["i"], experts=case["experts"],
                                     shared_experts=case["shared"], top_k=case["top_k"], max_moe_tokens=m,
                                     fp8=case["fp8"], score=case["score"], renormalize=True, routed_scale=2.5)
        else:
            s["sublayer"] = Sublayer()
    return s


# ------------------------------------------------------------- plain forms
def _plain_quantize(y):
    m, h = y.shape
    blocks = torch.nn.functional.pad(y, (0, _blocks(h) * BLOCK - h)).view(m, -1, BLOCK)
    amax = blocks.abs().amax(2).clamp(min=AMAX_FLOOR)
    values = (blocks * (E4M3_MAX / amax)[:, :, None]).view(m, -1)[:, :h].to(torch.float8_e4m3fn)
    return {"values": values, "scales": amax / E4M3_MAX}


def _plain_norm(inputs):
    r = inputs["x"].float() + inputs["residual"].float()
    y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * inputs["norm_weight"].float()
    return {"residual_out": r.bfloat16(), "output": y.bfloat16(), **_plain_quantize(y)}


def _plain_swiglu(inputs):
    gate, up = inputs["gate_up"].float().chunk(2, 1)
    return _plain_quantize(gate / (1.0 + torch.exp(-gate)) * up)


def _spread(scales, rows, cols):
    """[..., row blocks, column blocks] scales over [..., rows, cols]."""
    s = scales.repeat_interleave(BLOCK, -1)[..., :cols]
    return s.repeat_interleave(BLOCK, -2)[..., :rows, :]


def _plain_matmul(inputs, dtype):
    k = inputs["values"].shape[1]
    n = inputs["weight"].shape[0]
    a = inputs["values"].float() * inputs["scales"].repeat_interleave(BLOCK, 1)[:, :k]
    w = inputs["weight"].float() * _spread(inputs["weight_scales"], n, k)
    return {"output": (a @ w.t()).to(dtype)}


def _route(logits, bias, case):
    """(idx, weights) of the top_k experts: highest score (plus bias) first, ties to the lowest index."""
    if case["score"] == "softmax":
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    ranked = score if bias is None else score + bias
    idx = torch.sort(ranked, dim=1, descending=True, stable=True)[1][:, :case["top_k"]]
    w = score.gather(1, idx)
    return idx, w / w.sum(1, keepdim=True) * 2.5


def _plain_moe(inputs, case):
    x = inputs["x"].float()
    m, h = x.shape
    i, e, sh = case["i"], case["experts"], case["shared"]
    idx, w = _route(x @ inputs["router"].float().t(), inputs.get("bias"), case)
    every = torch.cat([idx, torch.arange(e, e + sh, device="cuda").expand(m, sh)], 1)
    weight = torch.cat([w, torch.ones(m, sh, device="cuda")], 1)
    flat = every.reshape(-1)
    if case["fp8"]:
        pick = lambda t: t.view(torch.uint8)[flat].view(torch.float8_e4m3fn).float()  # noqa: E731
        gate_up = pick(inputs["gate_up"]).view(-1, 2, i, h)
        gate_up *= _spread(inputs["gate_up_scales"][flat], i, h)
        down = pick(inputs["down"])
        down *= _spread(inputs["down_scales"][flat], h, i)
    else:
        gate_up = inputs["gate_up"][flat].float().view(-1, 2, i, h)
        down = inputs["down"][flat].float()
    rows = x.repeat_interleave(every.shape[1], 0)
    act = torch.matmul(gate_up.view(-1, 2 * i, h), rows[:, :, None])[:, :, 0]
    gate, up = act[:, :i], act[:, i:]
    act = gate / (1.0 + torch.exp(-gate)) * up
    y = torch.matmul(down, act[:, :, None])[:, :, 0].view(m, -1, h)
    return {"output": (y * weight[:, :, None]).sum(1).bfloat16(), "idx": idx.int(), "weights": w}


def run(state):
    case, inputs = state["case"], state["inputs"]
    op = case["op"]
    if own:
        s, outputs = state["sublayer"], state["outputs"]
        if op == "norm":
            return s.add_rms_norm(inputs, outputs, eps=EPS)
        if op == "quantize":
            return s.quantize(inputs, outputs)
        if op == "swiglu":
            return s.swiglu(inputs, outputs)
        if op == "matmul":
            return s.matmul(inputs, outputs)
        return s.moe(inputs, outputs)
    if op == "norm":
        return _plain_norm(inputs)
    if op == "quantize":
        return _plain_quantize(inputs["x"].float())
    if op == "swiglu":
        return _plain_swiglu(inputs)
    if op == "matmul":
        return _plain_matmul(inputs, state["outputs"]["output"].dtype)
    return _plain_moe(inputs, case)


# -------------------------------------------------------------------- work
def work(case):
    op, m = case["op"], case["m"]
    if op in ("norm", "quantize", "swiglu"):
        h = case["h"]
        eight = m * h + m * _blocks(h) * 4
        if op == "norm":
            return {"bytes": 4 * m * h * 2 + h * 2 + eight, "flops": 6 * m * h}
        return {"bytes": (2 if op == "swiglu" else 1) * m * h * 2 + eight, "flops": (6 if op == "swiglu" else 2) * m * h}
    if op == "matmul":
        n, k = case["n"], case["k"]
        out = 2 if case["out"] == "bf16" else 4
        return {"bytes": m * k + m * _blocks(k) * 4 + n * k + _blocks(n) * _blocks(k) * 4 + m * n * out,
                "flops": 2 * m * n * k}
    h, i, e, top = case["h"], case["i"], case["experts"], case["top_k"]
    reached = e * (1.0 - (1.0 - top / e) ** m) + case["shared"]     # experts that m tokens choose, expected
    per = 3 * i * h if case["fp8"] else 6 * i * h
    scales = 12 * _blocks(i) * _blocks(h) if case["fp8"] else 0
    return {"bytes": reached * (per + scales) + e * h * 2 + m * h * 4 + m * top * 8,
            "flops": 2 * m * (top + case["shared"]) * 3 * i * h + 2 * m * e * h}


# ------------------------------------------------- the definition in 64 bits
def _exact_blocks(y):
    m, h = y.shape
    values, scales = torch.empty_like(y), y.new_empty(m, _blocks(h))
    for b in range(_blocks(h)):
        part = y[:, b * BLOCK:(b + 1) * BLOCK]
        scales[:, b] = part.abs().max(1).values.clamp(min=AMAX_FLOOR) / 448.0
        values[:, b * BLOCK:(b + 1) * BLOCK] = part / scales[:, b, None]
    return {"values": values, "scales": scales}


def _exact_weight(values, scales):
    w = values.double()
    for r in range(scales.shape[0]):
        for c in range(scales.shape[1]):
            w[r * BLOCK:(r + 1) * BLOCK, c * BLOCK:(c + 1) * BLOCK] *= scales[r, c].double()
    return w


def exact(case, seed):
    inputs = prepare(case, seed)["inputs"]
    op = case["op"]
    if op == "norm":
        r = inputs["x"].double() + inputs["residual"].double()
        y = r / ((r * r).sum(1, keepdim=True) / r.shape[1] + EPS).sqrt() * inputs["norm_weight"].double()
        return {"residual_out": r, "output": y, **_exact_blocks(y)}
    if op == "quantize":
        return _exact_blocks(inputs["x"].double())
    if op == "swiglu":
        x = inputs["gate_up"].double()
        h = x.shape[1] // 2
        return _exact_blocks(x[:, :h] * torch.sigmoid(x[:, :h]) * x[:, h:])
    if op == "matmul":
        a = inputs["values"].double()
        for b in range(inputs["scales"].shape[1]):
            a[:, b * BLOCK:(b + 1) * BLOCK] *= inputs["scales"][:, b, None].double()
        return {"output": a @ _exact_weight(inputs["weight"], inputs["weight_scales"]).t()}
    x = inputs["x"].double()
    i, e, sh, top = case["i"], case["experts"], case["shared"], case["top_k"]
    logits = x @ inputs["router"].double().t()
    score = torch.softmax(logits, 1) if case["score"] == "softmax" else torch.sigmoid(logits)
    ranked = score + inputs["bias"].double() if "bias" in inputs else score
    idx = torch.argsort(ranked, dim=1, descending=True, stable=True)[:, :top]
    w = torch.take_along_dim(score, idx, 1)
    w = 2.5 * w / w.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for j in range(e + sh):
        if j < e:
            token, place = (idx == j).nonzero(as_tuple=True)
            share = w[token, place]
        else:
            token = torch.arange(x.shape[0], device="cuda")
            share = torch.ones_like(x[:, 0])
        if not token.numel():
            continue
        if case["fp8"]:
            gate = _exact_weight(inputs["gate_up"][j][:i], inputs["gate_up_scales"][j][0])
            up = _exact_weight(inputs["gate_up"][j][i:], inputs["gate_up_scales"][j][1])
            down = _exact_weight(inputs["down"][j], inputs["down_scales"][j])
        else:
            gate, up = inputs["gate_up"][j].double().chunk(2)
            down = inputs["down"][j].double()
        g = x[token] @ gate.t()
        y.index_add_(0, token, share[:, None] * ((g * torch.sigmoid(g) * (x[token] @ up.t())) @ down.t()))
    return {"output": y, "idx": None, "weights": w}

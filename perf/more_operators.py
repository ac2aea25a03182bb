"""Attention over a paged key-value cache, in its plain form and as the framework's calls.

The cache is cut into pages of `page` positions, [pages][kv_heads][page][head_dim] for the keys and again for the
values, in BF16 or in 8 bits (E4M3 values, one FP32 scale for each position and head).

* append  rotates queries and keys by their positions and writes keys and values into the cache, each token at its
          slot (page * page_size + offset; -1: a padding token, which is not written).
* decode  one new token of each sequence against that sequence's cache.
* prompt  several new tokens of each sequence, the last of the sequence: query i of n in a sequence of L positions
          stands at L - n + i and sees the positions up to its own, with a window only the last `window` of
          them and the first `sinks` of the sequence.

Outputs of decode and prompt: the attention's rows and the logarithm of each row's sum of exponentials; a row that
sees nothing has zeros and minus infinity.

`own` chooses the form: False runs elementary torch operations in 32 bits (the rotation's angles in 64), True the
package's Attention.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100     # an all-zero row gets this maximum, so that no scale is zero


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token's rotation and write, far into a sequence: latency
        {"name": "append_1", "op": "append", "m": 1, "heads": 40, "kv_heads": 8, "dim": 128, "page": 16, "fp8": False,
         "rotary": 128, "interleaved": False, "far": 1000000, "skip": False},
        # an odd number of tokens of many sequences, some of them padding, into an 8-bit cache; half of each head
        # is rotated, in neighbouring pairs
        {"name": "append_777", "op": "append", "m": 777, "heads": 16, "kv_heads": 2, "dim": 64, "page": 32, "fp8": True,
         "rotary": 32, "interleaved": True, "far": 30000, "skip": True},
        # a long prompt: the memory rate
        {"name": "append_8192", "op": "append", "m": 8192, "heads": 48, "kv_heads": 8, "dim": 128, "page": 64,
         "fp8": False, "rotary": 128, "interleaved": False, "far": 8192, "skip": False},
        # the first tokens of a chat with one user, where only latency counts
        {"name": "decode_1", "op": "decode", "b": 1, "length": 700, "heads": 40, "kv_heads": 8, "dim": 128, "page": 16,
         "fp8": False, "window": 0, "sinks": 0},
        # one user with a very long document: the work has to be split over the length
        {"name": "decode_1_long", "op": "decode", "b": 1, "length": 131072, "heads": 48, "kv_heads": 8, "dim": 128,
         "page": 64, "fp8": False, "window": 0, "sinks": 0},
        # a decode batch with lengths of every size: the memory rate
        {"name": "decode_64", "op": "decode", "b": 64, "length": 8192, "heads": 48, "kv_heads": 8, "dim": 128, "page": 64,
         "fp8": False, "window": 0, "sinks": 0},
        # an odd batch over an 8-bit cache
        {"name": "decode_37_8bit", "op": "decode", "b": 37, "length": 16001, "heads": 64, "kv_heads": 4, "dim": 128,
         "page": 32, "fp8": True, "window": 0, "sinks": 0},
        # a large batch in a layer with a short window and a few first tokens that stay visible; some rows are empty
        {"name": "decode_256_window", "op": "decode", "b": 256, "length": 4000, "heads": 32, "kv_heads": 4, "dim": 64,
         "page": 16, "fp8": False, "window": 512, "sinks": 4},
        # four proposed tokens of each of eight sequences, to be verified against long caches
        {"name": "prompt_verify", "op": "prompt", "b": 8, "queries": 4, "length": 32768, "heads": 32, "kv_heads": 4,
         "dim": 128, "page": 64, "fp8": False, "window": 0, "sinks": 0},
        # a whole prompt: the tensor rate
        {"name": "prompt_4096", "op": "prompt", "b": 1, "queries": 4096, "length": 4096, "heads": 48, "kv_heads": 8,
         "dim": 128, "page": 64, "fp8": False, "window": 0, "sinks": 0},
        # a long prompt of odd length in a layer with a window and first tokens that stay visible
        {"name": "prompt_window", "op": "prompt", "b": 1, "queries": 6001, "length": 6001, "heads": 32, "kv_heads": 4,
         "dim": 64, "page": 16, "fp8": False, "window": 1024, "sinks": 4},
        # the next chunks of ragged prompts over an 8-bit cache that holds what came before
        {"name": "prompt_chunks", "op": "prompt", "b": 3, "queries": 1024, "length": 8000, "heads": 40, "kv_heads": 8,
         "dim": 128, "page": 32, "fp8": True, "window": 0, "sinks": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "prompt", "prompt"])
    kv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "heads": kv * rng.randint(1, 8), "kv_heads": kv, "dim": rng.choice([64, 128, 128]),
         "page": rng.choice([16, 32, 64, 128]), "fp8": rng.random() < 0.4}
    if op == "append":
        c.update(m=_log(rng, 1, 8000), rotary=rng.choice([c["dim"], c["dim"] // 2]), interleaved=rng.random() < 0.5,
                 far=_log(rng, 10000, 1000000), skip=rng.random() < 0.3)
        return c
    if op == "decode":
        b = _log(rng, 1, 256)
        length = _log(rng, 1, min(131072, 500000 // b))
    else:
        b = _log(rng, 1, 8)
        queries = _log(rng, 2, 4000)
        # as many positions as keep the plain form's scores within those of the largest case
        length = _log(rng, queries, max(queries, min(32768, 600000000 // (b * queries * c["heads"]))))
        queries = min(queries, 600000000 // (b * length * c["heads"]))
        c["queries"] = max(2, queries)
        length = max(length, c["queries"])
    windowed = rng.random() < 0.4
    c.update(b=b, length=length, window=_log(rng, 1, 4096) if windowed else 0, sinks=rng.randint(0, 8) if windowed else 0)
    return c


def _ragged(case):
    """(lengths, queries) of the case's sequences: the first has the most, the others any number; in a large
    batch some are empty."""
    b, rng = case["b"], random.Random(case["b"] * 1000003 + case["length"])
    lengths = [case["length"]] + [rng.randint(1, case["length"]) for _ in range(b - 1)]
    if b >= 32:
        lengths[7] = lengths[b - 1] = 0
    if case["op"] == "decode":
        return lengths, [1] * b
    most = case["queries"]
    if most <= 16:
        return lengths, [most] * b
    return lengths, [most] + [rng.randint(1, min(most, n)) for n in lengths[1:]]


# ------------------------------------------------------------------ inputs
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _cache(g, case, pages):
    """Keys with a few channels that are larger, as after a rotation of real projections, and values."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    gain = 1.0 + 2.0 * (torch.rand(case["kv_heads"], 1, case["dim"], generator=g, device="cuda") < 0.05)
    k, v = _randn(g, *shape) * gain, _randn(g, *shape)
    if not case["fp8"]:
        return {"k_cache": k.bfloat16(), "v_cache": v.bfloat16()}
    out = {}
    for name, x in (("k", k), ("v", v)):
        values, out[name + "_scales"] = _plain_quantize(x * (0.5 + torch.rand(*shape[:3], 1, generator=g, device="cuda")))
        out[name + "_cache"] = values
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    hq, kv, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    s = {"case": case}
    if case["op"] == "append":
        m = case["m"]
        # the tokens' places: pages in no order; the last page is nobody's
        pages = m // page + 2
        slots = torch.randperm((pages - 1) * page, generator=g, device="cuda")[:m].int()
        if case["skip"]:
            slots[m // 3::5] = -1
        qkv = _randn(g, m, (hq + 2 * kv) * d).bfloat16()
        split = qkv.view(m, hq + 2 * kv, d).split([hq, kv, kv], 1)   # heads of one projection's rows
        positions = torch.randint(0, case["far"], (m,), generator=g, device="cuda").int()
        s["inputs"] = {"q": split[0], "k": split[1], "v": split[2], "positions": positions, "slots": slots}
        s["outputs"] = {"q_out": torch.empty(m, hq, d, dtype=torch.bfloat16, device="cuda"), **_cache(g, case, pages)}
    else:
        lengths, queries = _ragged(case)
        b, t = case["b"], sum(queries)
        width = -(-case["length"] // page)
        own_pages = [-(-n // page) for n in lengths]
        pages = sum(own_pages) + 1
        order = torch.randperm(pages, generator=g, device="cuda").int()
        at = torch.tensor([0] + own_pages, device="cuda").cumsum(0)[:-1]
        used = torch.arange(width, device="cuda")[None, :] < torch.tensor(own_pages, device="cuda")[:, None]
        index = (at[:, None] + torch.arange(width, device="cuda")[None, :]).clamp(max=pages - 1)
        s["inputs"] = {"q": (1.2 * _randn(g, t, hq, d)).bfloat16(), **_cache(g, case, pages),
                       "pages": torch.where(used, order[index], 0).int(),
                       "lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda")}
        if case["op"] == "prompt":
            s["inputs"]["q_starts"] = torch.tensor([0] + queries, device="cuda").cumsum(0).int()
        s["outputs"] = {"output": torch.empty(t, hq, d, dtype=torch.bfloat16, device="cuda"),
                        "lse": torch.empty(t, hq, dtype=torch.float32, device="cuda")}
    if own:
        from mhc_residual_boundary_gb300 import Attention
        rotary = case.get("rotary", 0)
        s["attention"] = Attention(heads=hq, kv_heads=kv, head_dim=d, page_size=page, fp8=case["fp8"], rotary_dim=rotary,
                                   theta=500000.0, interleaved=case.get("interleaved", False))
    return s


# ------------------------------------------------------------- plain forms
def _plain_quantize(x):
    amax = x.abs().amax(-1).clamp(min=AMAX_FLOOR)
    return (x * (E4M3_MAX / amax)[..., None]).to(torch.float8_e4m3fn), amax / E4M3_MAX


def _plain_rotate(x, positions, case):
    r = case["rotary"]
    turn = 500000.0 ** (torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / -r)
    angle = positions.double()[:, None] * turn
    c, s = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    if case["interleaved"]:
        a, b = x[..., :r:2], x[..., 1:r:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_write(cache, rows, slots, page):
    """Rows [m][kv_heads][...] of the cache [pages][kv_heads][page][...]; a token without a slot rewrites what the
    last place, which is nobody's, holds."""
    live = slots >= 0
    spot = torch.where(live, slots, cache.shape[0] * page - 1).long()
    where, offset = spot // page, spot % page
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    rows = rows.view(torch.uint8) if rows.dtype == torch.float8_e4m3fn else rows
    keep = live.view(-1, *([1] * (rows.dim() - 1)))
    raw[where, :, offset] = torch.where(keep, rows, raw[where, :, offset])


def _plain_append(inputs, outputs, case):
    positions, slots, page = inputs["positions"], inputs["slots"], case["page"]
    k, v = _plain_rotate(inputs["k"].float(), positions, case), inputs["v"].float()
    if case["fp8"]:
        k, k_scales = _plain_quantize(k)
        v, v_scales = _plain_quantize(v)
        _plain_write(outputs["k_scales"], k_scales, slots, page)
        _plain_write(outputs["v_scales"], v_scales, slots, page)
    else:
        k, v = k.bfloat16(), v.bfloat16()
    _plain_write(outputs["k_cache"], k, slots, page)
    _plain_write(outputs["v_cache"], v, slots, page)
    return {**outputs, "q_out": _plain_rotate(inputs["q"].float(), positions, case).bfloat16()}


def _plain_gather(inputs, name):
    """A cache's rows in the sequences' order: [b][kv_heads][positions][dim] in 32 bits."""
    pages = inputs["pages"].long()
    x = inputs[name + "_cache"]
    if x.dtype == torch.float8_e4m3fn:
        x = x.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
        x = x * inputs[name + "_scales"][pages][..., None]
    else:
        x = x[pages].float()
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(inputs, case):
    q, lengths = inputs["q"], inputs["lengths"].long()
    t, hq, d = q.shape
    b, kv = case["b"], case["kv_heads"]
    most = case.get("queries", 1)
    starts = inputs["q_starts"].long() if "q_starts" in inputs else torch.arange(b + 1, device="cuda")
    count = starts[1:] - starts[:-1]
    i = torch.arange(most, device="cuda")
    rows = (starts[:-1, None] + i).clamp(max=t - 1)
    padded = q[rows].float().view(b, most, kv, hq // kv, d).permute(0, 2, 3, 1, 4)       # [b][kv][group][most][d]
    k, v = _plain_gather(inputs, "k"), _plain_gather(inputs, "v")
    scores = torch.matmul(padded.flatten(2, 3), k.transpose(2, 3)).view(b, kv, hq // kv, most, -1) / math.sqrt(d)
    at = (lengths - count)[:, None] + i
    j = torch.arange(k.shape[2], device="cuda")
    seen = (j <= at[..., None]) & (j < lengths[:, None, None]) & (i < count[:, None])[..., None]
    if case["window"]:
        seen &= (j > at[..., None] - case["window"]) | (j < case["sinks"])
    scores = scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    scores = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.flatten(2, 3), v).view(b, kv, hq // kv, most, d)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 3, 1, 2, 4).reshape(b, most, hq, d)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(b, most, hq)
    token = torch.arange(t, device="cuda")
    sequence = torch.searchsorted(starts, token, right=True) - 1
    place = token - starts[sequence]
    return {"output": out[sequence, place].bfloat16(), "lse": lse[sequence, place]}


def run(state):
    case, inputs, outputs = state["case"], state["inputs"], state["outputs"]
    if own:
        if case["op"] == "append":
            return state["attention"].append(inputs, outputs)
        return state["attention"].attend(inputs, outputs, window=case["window"], sinks=case["sinks"])
    if case["op"] == "append":
        return _plain_append(inputs, outputs, case)
    return _plain_attend(inputs, case)


# -------------------------------------------------------------------- work
def _seen(at, window, sinks):
    """Positions that the query at position `at` sees."""
    if at < 0:
        return 0
    if not window or at < window:
        return at + 1
    return window + min(sinks, at + 1 - window)


def work(case):
    hq, kv, d = case["heads"], case["kv_heads"], case["dim"]
    row = d + 4 if case["fp8"] else 2 * d
    if case["op"] == "append":
        m = case["m"]
        return {"bytes": m * (hq * d * 4 + 2 * kv * (d * 2 + row) + 8), "flops": 3 * m * (hq + kv) * case["rotary"]}
    lengths, queries = _ragged(case)
    positions = pairs = 0
    for n, count in zip(lengths, queries):
        pairs += sum(_seen(n - count + i, case["window"], case["sinks"]) for i in range(count))
        # positions that some query of the sequence sees
        first = max(0, n - count + 1 - case["window"]) if case["window"] else 0
        positions += n - first + min(case["sinks"], first)
    t = sum(queries)
    return {"bytes": positions * kv * 2 * row + t * hq * (4 * d + 4), "flops": 4 * d * hq * pairs}


# ------------------------------------------------- the definition in 64 bits
def _exact_rotate(x, positions, case):
    r, y = case["rotary"], x.double()
    out = y.clone()
    for i in range(r // 2):
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
        angle = positions.double() * 500000.0 ** (-2.0 * i / r)
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        out[:, :, first] = y[:, :, first] * c - y[:, :, second] * s
        out[:, :, second] = y[:, :, second] * c + y[:, :, first] * s
    return out


def _exact_append(inputs, outputs, case):
    result = {name: x.double() for name, x in outputs.items()}
    result["q_out"] = _exact_rotate(inputs["q"], inputs["positions"], case)
    live = (inputs["slots"] >= 0).nonzero()[:, 0]
    where, offset = inputs["slots"][live].long() // case["page"], inputs["slots"][live].long() % case["page"]
    for name, rows in (("k", _exact_rotate(inputs["k"], inputs["positions"], case)), ("v", inputs["v"].double())):
        rows = rows[live]
        if case["fp8"]:
            scales = rows.abs().max(2).values.clamp(min=AMAX_FLOOR) / 448.0
            result[name + "_scales"][where, :, offset] = scales
            rows = rows / scales[:, :, None]
        result[name + "_cache"][where, :, offset] = rows
    return result


def exact(case, seed):
    s = prepare(case, seed)
    inputs, page = s["inputs"], case["page"]
    if case["op"] == "append":
        return _exact_append(inputs, s["outputs"], case)
    lengths, queries = _ragged(case)
    group, window = case["heads"] // case["kv_heads"], case["window"]
    out = torch.zeros(s["outputs"]["output"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    begin = 0
    for n, count, table in zip(lengths, queries, inputs["pages"]):
        end = begin + count
        for h in range(case["kv_heads"] if n else 0):
            chosen = table[:-(-n // page)].long()
            k, v = (inputs[x][chosen, h].flatten(0, 1)[:n].double() for x in ("k_cache", "v_cache"))
            if case["fp8"]:
                k = k * inputs["k_scales"][chosen, h].flatten()[:n, None].double()
                v = v * inputs["v_scales"][chosen, h].flatten()[:n, None].double()
            behind = torch.arange(n - count, n, device="cuda")[:, None] - torch.arange(n, device="cuda")
            hidden = behind < 0
            if window:
                hidden |= (behind >= window) & (torch.arange(n, device="cuda") >= case["sinks"])
            for g in range(h * group, (h + 1) * group):
                scores = inputs["q"][begin:end, g].double() @ k.t() * case["dim"] ** -0.5
                scores[hidden] = -math.inf
                lse[begin:end, g] = torch.logsumexp(scores, 1)
                out[begin:end, g] = torch.softmax(scores, 1).nan_to_num(0.0) @ v
        begin = end
    return {"output": out, "lse": lse}

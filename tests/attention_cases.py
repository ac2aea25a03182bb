"""Inputs and the 64-bit definition for the attention tests.

Tolerances, from the arithmetic (w the softmax weights, sum w = 1):
* a score x is a sum of exact products in FP32: off by at most 2^-20 of S = scale
  * sum |q k|, and its exponential and the sums of weights by 2^-20 of themselves
  (rounding of the exponent's argument, the exponential's own error, the sums), so
  a weight by 2 (S + 2) 2^-20 of itself;
* the weight is rounded for the matrix product: to BF16 (2^-8 of itself) in calls
  with q_starts or more than 16 heads a kv head, to FP16 over an 8-bit cache in
  the others (2^-11 of itself, or 2^-25 of the largest below FP16's normals), to two
  BF16 pieces (2^-16) over a BF16 one;
* queries over an 8-bit cache have a power of two taken off each row: in FP16 that
  changes an element by at most 2^-25 of the row's largest, in two E4M3 pieces (calls
  with q_starts or more than 16 heads a kv head) by at most 2^-17 of it: S takes the
  elements with that over 2^-20 added;
* the output is rounded to BF16: half an ulp of what is rounded, which is off itself, and
  so may lie in the binade above;
so an output is off by at most e + half an ulp at |out| + e, with
e = (rounding + 2 (S + 2) 2^-20) * sum w |v|.
* lse is off by at most (S + |lse| + 2) 2^-20.
"""
import torch

F8, BF16, F32, I32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32
STEPS = 2.0 ** -20


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def make_cache(g, pages, kv, page, d, fp8):
    k, v = randn(g, pages, kv, page, d), randn(g, pages, kv, page, d)
    if not fp8:
        return {"k_cache": k.to(BF16), "v_cache": v.to(BF16)}
    out = {}
    for name, x in (("k", k), ("v", v)):
        x = x * (0.25 + 2 * torch.rand(pages, kv, page, 1, generator=g, device="cuda"))
        scale = x.abs().amax(-1) / 448
        out[name + "_cache"] = (x / scale[..., None]).clamp(-448, 448).to(F8)
        out[name + "_scales"] = scale
    return out


def make_inputs(seed, *, lengths, queries=None, heads, kv, d, page, fp8, spare=3, size=1.0):
    """attend's inputs for sequences of these lengths (queries None: one each), pages in no order."""
    g = gen(seed)
    need = [-(-n // page) for n in lengths]
    pages, width = sum(need) + spare, max(need + [1])
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lengths), width), -1, dtype=I32, device="cuda")   # no page behind a sequence's last
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    t = len(lengths) if queries is None else sum(queries)
    inputs = {"q": (size * randn(g, t, heads, d)).to(BF16), **make_cache(g, pages, kv, page, d, fp8), "pages": table,
              "lengths": torch.tensor(lengths, dtype=I32, device="cuda")}
    if queries is not None:
        inputs["q_starts"] = torch.tensor([0] + queries, device="cuda").cumsum(0).int()
    return inputs


def rows_of(inputs, name, s, n, page):
    """Positions [kv][n][d] of sequence s in 64 bits."""
    chosen = inputs["pages"][s, :-(-n // page)].long()
    x = inputs[name + "_cache"]
    x = x.view(torch.uint8)[chosen].view(F8).double() if x.dtype == F8 else x[chosen].double()
    if name + "_scales" in inputs:
        x = x * inputs[name + "_scales"][chosen].double()[..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def seen_by(at, window, sinks):
    j = torch.arange(max(at + 1, 0), device="cuda")
    return j[(j > at - window) | (j < sinks)] if window else j


def define(inputs, *, window=0, sinks=0, scale=None, page, gone=()):
    """The definition, query by query over the positions it sees: output, lse, sum w |v| and S.  gone: (sequence,
    page of it) whose positions are not there."""
    q = inputs["q"].double()
    t, heads, d = q.shape
    kv = inputs["k_cache"].shape[1]
    scale = d ** -0.5 if scale is None else scale
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((t, heads), -float("inf"), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(lse)
    lengths = inputs["lengths"].tolist()
    starts = inputs["q_starts"].tolist() if "q_starts" in inputs else list(range(t + 1))
    for s, n in enumerate(lengths):
        if n == 0 or starts[s] == starts[s + 1]:
            continue
        k, v = rows_of(inputs, "k", s, n, page), rows_of(inputs, "v", s, n, page)
        for i in range(starts[s], starts[s + 1]):
            seen = seen_by(n - (starts[s + 1] - i), window, sinks)
            for hole in (g for r, g in gone if r == s):
                seen = seen[seen // page != hole]
            if not len(seen):
                continue
            qi = q[i].view(kv, heads // kv, d)
            x = scale * torch.einsum("kgd,knd->kgn", qi, k[:, seen])
            w = torch.softmax(x, -1)
            out[i] = torch.einsum("kgn,knd->kgd", w, v[:, seen]).reshape(heads, d)
            mag[i] = torch.einsum("kgn,knd->kgd", w, v[:, seen].abs()).reshape(heads, d)
            lse[i] = torch.logsumexp(x, -1).flatten()
            near = qi.abs() + query_rounding(inputs) / STEPS * qi.abs().amax(-1, keepdim=True)
            size[i] = (scale * torch.einsum("kgd,knd->kgn", near, k[:, seen].abs())).amax(-1).flatten()
    return out, lse, mag, size


def weight_rounding(inputs):
    heads, kv = inputs["q"].shape[1], inputs["k_cache"].shape[1]
    if "q_starts" in inputs or heads // kv > 16:
        return 2.0 ** -8
    return 2.0 ** -11 if "k_scales" in inputs else 2.0 ** -16


def query_rounding(inputs):
    if "k_scales" not in inputs:
        return 0.0
    return 2.0 ** -17 if weight_rounding(inputs) == 2.0 ** -8 else 2.0 ** -25


def half_ulp_bf16(x):
    return torch.ldexp(torch.ones_like(x), torch.frexp(x)[1] - 9)


def check(outputs, inputs, *, page, window=0, sinks=0, scale=None, want=None):
    out, lse, mag, size = want or define(inputs, window=window, sinks=sinks, scale=scale, page=page)
    t = out.shape[0] if "q_starts" not in inputs else int(inputs["q_starts"][-1])
    got = outputs["output"][:t].double()
    out, lse, mag, size = out[:t], lse[:t], mag[:t], size[:t]
    # FP16 weights below the normals: 2^-25 of the largest weight for each position, which is at most twice 1 / sum
    small = 0.0
    if "k_scales" in inputs and weight_rounding(inputs) == 2.0 ** -11:
        n = inputs["lengths"].double().amax()
        small = 2.0 ** -24 * n * mag.amax(-1, keepdim=True)
    before = (weight_rounding(inputs) + 2 * (size + 2)[..., None] * STEPS) * mag + small + 1e-38
    limit = half_ulp_bf16(out.abs() + before) + before
    bad = ~((got - out).abs() <= limit)
    assert not bad.any(), ("output", int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), out[bad][:4].tolist())
    if "lse" in outputs:
        got = outputs["lse"][:t].double()
        empty = lse == -float("inf")
        assert (got[empty] == -float("inf")).all()
        bad = ~((got - lse).abs() <= (size + lse.abs() + 2) * STEPS) & ~empty
        assert not bad.any(), ("lse", bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), lse[bad][:4].tolist())

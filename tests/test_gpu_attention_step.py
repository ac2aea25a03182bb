"""The attention operators together, as they are used: prompts appended and attended, then steps of one token a
sequence, called and captured; and examples/decoder_step.py with its attention.  Each call is checked against the
definition in 64 bits of what it was given; a prompt's rows, too, against the same tokens one at a time."""
import pytest
import torch

from attention_cases import BF16, F8, I32, check, define, gen, randn
from test_gpu_append import check_bf16, check_fp8, rotate
from test_gpu_decoder_step import example  # noqa: F401  (a fixture)
from test_gpu_sublayer import check_product, check_quantized

pytestmark = pytest.mark.gpu


class Serving:
    """Sequences of random tokens in a paged cache: `step` appends the next `counts` tokens of each and attends."""

    def __init__(self, a, counts, capacity, seed):
        self.a, self.g, self.s = a, gen(seed), len(counts)
        self.page, self.width = a.page_size, -(-capacity // a.page_size)
        self.cache = a.empty_cache(self.s * self.width)
        for x in self.cache.values():
            x.view(torch.uint8).fill_(0xff)   # NaN: what nothing was written to
        self.pages = torch.randperm(self.s * self.width, generator=self.g, device="cuda").int().view(self.s, -1)
        self.lengths = torch.zeros(self.s, dtype=I32, device="cuda")

    def tokens(self, counts):
        t, heads, kv, d = sum(counts), self.a.heads, self.a.kv_heads, self.a.head_dim
        packed = randn(self.g, t, heads + 2 * kv, d).to(BF16)
        return packed.split([heads, kv, kv], 1)

    def places(self, counts):
        """positions, slots and the lengths afterwards."""
        seq = torch.repeat_interleave(torch.arange(self.s, device="cuda"), torch.tensor(counts, device="cuda"))
        at = torch.cat([torch.arange(n, device="cuda") for n in counts]) + self.lengths[seq]
        slots = self.pages[seq, (at // self.page).long()] * self.page + at % self.page
        return at.int(), slots.int(), self.lengths + torch.tensor(counts, dtype=I32, device="cuda")

    def inputs(self, q, lengths, counts=None):
        out = {"q": q, "pages": self.pages, "lengths": lengths, **self.cache}
        if counts:
            out["q_starts"] = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
        return out


def check_stored(serving, name, x, positions, slots, frequencies):
    page, d = serving.page, x.shape[-1]
    want, mag = rotate(x, positions, frequencies, d, False) if name == "k" else (x.double(), x.double().abs())
    where, offset = slots.long() // page, slots.long() % page
    stored = serving.cache[name + "_cache"]
    if stored.dtype == F8:
        check_fp8(stored.view(torch.uint8)[where, :, offset].view(F8).float(), serving.cache[name + "_scales"][where, :, offset],
                  want, mag)
    else:
        check_bf16(stored[where, :, offset], want, mag)


@pytest.mark.parametrize("heads, kv, d, page, fp8, window, sinks", [
    (8, 2, 128, 16, False, 0, 0), (8, 2, 128, 64, True, 0, 0), (12, 4, 64, 32, False, 100, 3), (40, 2, 64, 128, True, 0, 0)])
def test_prompts_then_steps(heads, kv, d, page, fp8, window, sinks):
    from mhc_residual_boundary_gb300 import Attention
    a = Attention(heads=heads, kv_heads=kv, head_dim=d, page_size=page, fp8=fp8, rotary_dim=d)
    frequencies = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    serving = Serving(a, [0] * 4, 700, 3)
    kw = {"window": window, "sinks": sinks}
    # prompts, then a chunk for two of the sequences
    for counts in ([300, 1, 17, 140], [200, 0, 130, 0]):
        q, k, v = serving.tokens(counts)
        positions, slots, lengths = serving.places(counts)
        rotated, _ = rotate(q, positions, frequencies, d, False)
        a.append({"q": q, "k": k, "v": v, "positions": positions, "slots": slots}, {"q_out": q, **serving.cache})
        assert ((q.double() - rotated).abs() <= 2.0 ** -8 * rotated.abs() + 1e-4).all()
        check_stored(serving, "k", k, positions, slots, frequencies)
        check_stored(serving, "v", v, positions, slots, frequencies)
        inputs = serving.inputs(q, lengths, counts)
        check(a.attend(inputs, a.empty_outputs(sum(counts)), **kw), inputs, page=page, window=window, sinks=sinks)
        serving.lengths = lengths
    a.check_errors()
    # steps: one token of each sequence, in a graph whose inputs change between replays
    q, k, v = (x.clone() for x in serving.tokens([1] * 4))
    positions, slots, lengths = serving.places([1] * 4)
    rotated, out = torch.empty_like(q), a.empty_outputs(4)

    def step():
        a.append({"q": q, "k": k, "v": v, "positions": positions, "slots": slots}, {"q_out": rotated, **serving.cache})
        a.attend(serving.inputs(rotated, lengths), out, **kw)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(page + 3):   # over the end of a page
        for x, y in zip((q, k, v), serving.tokens([1] * 4)):
            x.copy_(y)
        for x, y in zip((positions, slots, lengths), serving.places([1] * 4)):
            x.copy_(y)
        graph.replay()
        inputs = serving.inputs(rotated, lengths)
        check(out, inputs, page=page, window=window, sinks=sinks)
        check_stored(serving, "k", k, positions, slots, frequencies)
        serving.lengths = lengths.clone()
    a.check_errors()


def test_a_prompt_is_its_tokens_one_at_a_time():
    """Both are within their tolerances of the definition over the same cache."""
    from mhc_residual_boundary_gb300 import Attention
    a = Attention(heads=8, kv_heads=2, rotary_dim=128)
    serving = Serving(a, [0], 200, 5)
    q, k, v = serving.tokens([150])
    positions, slots, lengths = serving.places([150])
    a.append({"q": q, "k": k, "v": v, "positions": positions, "slots": slots}, {"q_out": q, **serving.cache})
    whole = serving.inputs(q, lengths, [150])
    want = define(whole, page=64)
    check(a.attend(whole, a.empty_outputs(150)), whole, page=64, want=want)
    # the same cache, as 150 sequences of 1, 2, ... positions
    many = {"q": q, "pages": serving.pages.expand(150, -1).contiguous(), "lengths": positions + 1, **serving.cache}
    check(a.attend(many, a.empty_outputs(150)), many, page=64, want=want)
    a.check_errors()


@pytest.mark.parametrize("m, fp8", [(1, False), (13, True), (32, False)])
def test_decoder_step(example, m, fp8):  # noqa: F811
    kw = dict(hidden=1024, tp=2, mlp=1280, intermediate=384, experts=16, shared_experts=1, top_k=4, vocab=2056, seed=m)
    s = example.DecoderStep(m, **kw, context=190, heads=8, kv_heads=2, fp8_cache=fp8)
    other = s.start["partials"][1].clone()
    first = s.step().clone()
    s.check_errors()
    frequencies = [10000.0 ** (-2.0 * i / 128) for i in range(64)]

    def checked():
        check_quantized(s.in8, s.attention_in.double())
        check_product(s.qkv_out["output"], {"values": s.in8["values"], "scales": s.in8["scales"], "weight": s.qkv[0],
                                            "weight_scales": s.qkv[1]})
        check_bf16(s.q_out, *rotate(s.q, s.positions, frequencies, 128, False))
        inputs = {"q": s.q_out, "pages": s.pages, "lengths": s.lengths, **s.cache}
        check(s.attended, inputs, page=64)
        check_quantized(s.attended8, s.attended["output"].view(m, -1).double())
        check_product(s.start["partials"][0], {"values": s.attended8["values"], "scales": s.attended8["scales"],
                                               "weight": s.o[0], "weight_scales": s.o[1]})
        assert torch.equal(s.start["partials"][1], other)
        assert torch.isfinite(s.logits["output"]).all()
    checked()
    graph = s.capture()
    s.logits["output"].zero_()
    graph.replay()
    assert torch.equal(s.logits["output"], first)
    for _ in range(3):   # over the end of a page
        s.advance()
        s.attention_in.copy_(s.randn(m, 1024))
        graph.replay()
        checked()
    s.check_errors()

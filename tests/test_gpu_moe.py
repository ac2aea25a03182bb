"""The MoE layer for a few tokens against its definition in 64 bits.

Tolerance of the output, from the arithmetic: the FP32 sums of the two
products are within 2^-20 of the sum of their terms' magnitudes; x enters
exactly but for values under 2^-13 of their row's largest, which are off by at
most 2^-23 of it; h is held to 12 bits (8-bit weights; off by 2^-12 of itself
or 2^-22 of its block's largest) or 16 (BF16 weights); an error of g or u
reaches h through silu, whose slope is at most 1.1; a routing weight is off by
the logits' error (2^-20 of the sum of their terms' magnitudes, twice: the
score and the scores' sum) and 2^-20 of itself; and the BF16 output adds half
an ulp.  The chosen experts must be equal.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

F8, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
STEPS = 2.0 ** -20


def blocks(n):
    return (n + 127) // 128


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


class Case:
    def __init__(self, m, h, i, experts, shared, top_k, fp8, score="softmax", renormalize=True, router_f32=False,
                 bias=False, scale=1.0, seed=0):
        if not torch.cuda.is_available():
            pytest.skip("needs a GPU")
        self.__dict__.update(m=m, h=h, i=i, e=experts, s=shared, k=top_k, fp8=fp8, score=score,
                             renormalize=renormalize, scale=scale)
        g = gen(seed + 7 * m + h + i + experts)
        every = experts + shared
        router = randn(g, experts, h) / h ** 0.5
        self.inputs = {"x": (randn(g, m, h) * (1 + 20 * (torch.rand(h, generator=g, device="cuda") < 0.02))).bfloat16(),
                       "router": router if router_f32 else router.bfloat16()}
        if bias:
            self.inputs["bias"] = 0.1 * randn(g, experts)
        if fp8:
            self.inputs["gate_up"] = (100 * randn(g, every, 2 * i, h)).clamp(-448, 448).to(F8)
            self.inputs["down"] = (100 * randn(g, every, h, i)).clamp(-448, 448).to(F8)
            self.inputs["gate_up_scales"] = ((0.5 + torch.rand(every, 2, blocks(i), blocks(h), generator=g,
                                                               device="cuda")) / (100 * h ** 0.5))
            self.inputs["down_scales"] = ((0.5 + torch.rand(every, blocks(h), blocks(i), generator=g, device="cuda"))
                                          / (100 * i ** 0.5))
        else:
            self.inputs["gate_up"] = (randn(g, every, 2 * i, h) / h ** 0.5).bfloat16()
            self.inputs["down"] = (randn(g, every, h, i) / i ** 0.5).bfloat16()
        from mhc_residual_boundary_gb300 import Sublayer
        self.layer = Sublayer(hidden=h, intermediate=i, experts=experts, shared_experts=shared, top_k=top_k,
                              max_moe_tokens=m, fp8=fp8, score=score, renormalize=renormalize, routed_scale=scale,
                              router_f32=router_f32)

    def run(self):
        out = self.layer.empty_outputs("moe", self.m)
        out["output"].fill_(float("nan"))
        out["idx"].fill_(-1)
        return self.layer.moe(self.inputs, out)

    def weights_of(self, j):
        """(gate, up, down) of expert j in 64 bits."""
        gate, up = self.inputs["gate_up"][j].double().view(2, self.i, self.h)
        down = self.inputs["down"][j].double()
        if self.fp8:
            def spread(s, rows, cols):
                return s.double().repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
            gs = self.inputs["gate_up_scales"][j]
            gate, up = gate * spread(gs[0], self.i, self.h), up * spread(gs[1], self.i, self.h)
            down = down * spread(self.inputs["down_scales"][j], self.h, self.i)
        return gate, up, down

    def check(self, out, rows=None):
        rows = list(range(self.m)) if rows is None else rows
        x = self.inputs["x"][rows].double()
        router = self.inputs["router"].double()
        logits = x @ router.t()
        logit_err = STEPS * (x.abs() @ router.abs().t()).amax(1)
        score = torch.softmax(logits, 1) if self.score == "softmax" else torch.sigmoid(logits)
        ranked = score + self.inputs["bias"].double() if "bias" in self.inputs else score
        idx = torch.argsort(ranked, dim=1, descending=True, stable=True)[:, :self.k]
        w = score.gather(1, idx)
        if self.renormalize:
            w = w / w.sum(1, keepdim=True)
        w = w * self.scale
        assert torch.equal(out["idx"][rows].long(), idx)
        w_err = 2 * logit_err + STEPS
        assert ((out["weights"][rows].double() - w).abs() <= w_err[:, None] * w).all()
        y, bound = torch.zeros_like(x), torch.zeros_like(x)
        for j in range(self.e + self.s):
            if j < self.e:
                token, place = (idx == j).nonzero(as_tuple=True)
                share, share_err = w[token, place], w_err[token]
            else:
                token = torch.arange(len(rows), device="cuda")
                share, share_err = torch.ones(len(rows), device="cuda").double(), torch.zeros(len(rows), device="cuda")
            if not len(token):
                continue
            gate, up, down = self.weights_of(j)
            xt = x[token]
            small = 2.0 ** -23 * xt.abs().amax(1, keepdim=True)
            gv, uv = xt @ gate.t(), xt @ up.t()
            g_err = STEPS * (xt.abs() @ gate.abs().t()) + small * gate.abs().sum(1)
            u_err = STEPS * (xt.abs() @ up.abs().t()) + small * up.abs().sum(1)
            silu = gv * torch.sigmoid(gv)
            hv = silu * uv
            pad = torch.nn.functional.pad(hv.abs(), (0, blocks(self.i) * 128 - self.i)).view(len(token), -1, 128)
            top = pad.amax(2).repeat_interleave(128, 1)[:, :self.i]
            h_err = 1.1 * uv.abs() * g_err + silu.abs() * u_err + STEPS * hv.abs()
            h_err = h_err + (2.0 ** -12 * hv.abs() + 2.0 ** -22 * top if self.fp8 else 2.0 ** -16 * hv.abs())
            part = hv @ down.t()
            size = hv.abs() @ down.abs().t()
            y.index_add_(0, token, share[:, None] * part)
            bound.index_add_(0, token, share[:, None] * (h_err @ down.abs().t() + STEPS * size
                                                         + share_err[:, None] * size))
        bound = bound + torch.ldexp(torch.ones_like(y), torch.frexp(y.abs() + bound)[1] - 9)
        off = (out["output"][rows].double() - y).abs()
        assert (off <= bound).all(), ((off / bound).max().item(), (off > bound).nonzero()[:4].tolist())


@pytest.mark.parametrize("m", [1, 2, 8, 9, 17, 32])
@pytest.mark.parametrize("h,i,experts,shared,top_k", [(16, 16, 1, 0, 1), (256, 128, 8, 0, 2), (272, 144, 4, 1, 4),
                                                      (1024, 512, 16, 2, 8), (512, 1040, 40, 0, 1)])
@pytest.mark.parametrize("fp8", [True, False])
def test_moe(m, h, i, experts, shared, top_k, fp8):
    c = Case(m, h, i, experts, shared, top_k, fp8)
    c.check(c.run())
    c.layer.check_errors()


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("options", [
    {"score": "sigmoid", "bias": True, "scale": 2.5}, {"renormalize": False}, {"router_f32": True, "bias": True},
    {"score": "sigmoid", "renormalize": False, "router_f32": True}])
def test_routing_options(fp8, options):
    c = Case(6, 264 if not fp8 else 272, 136 if not fp8 else 144, 24, 1, 6, fp8, **options)
    c.check(c.run())


# the widest of each size, and sizes that split every way over the CTAs
@pytest.mark.parametrize("m,h,i,experts,shared,top_k,fp8", [
    (32, 128, 16, 512, 8, 16, True), (3, 5120, 2048, 8, 1, 2, True), (1, 6144, 1024, 4, 0, 1, False),
    (32, 16384, 16, 2, 0, 1, True), (2, 128, 16384, 2, 0, 2, True), (31, 640, 384, 300, 3, 7, False)])
def test_moe_sizes(m, h, i, experts, shared, top_k, fp8):
    c = Case(m, h, i, experts, shared, top_k, fp8)
    c.check(c.run())


@pytest.mark.parametrize("fp8", [True, False])
def test_fewer_tokens_than_the_capacity_and_all_on_one_expert(fp8):
    c = Case(32, 256, 256, 16, 0, 2, fp8, bias=True)
    c.inputs["bias"].zero_()
    c.inputs["bias"][11], c.inputs["bias"][3] = 4.0, 2.0
    c.check(c.run())
    full = c.inputs["x"]
    for m in (1, 13):
        c.m, c.inputs["x"] = m, full[:m].contiguous()
        out = c.run()
        assert (out["idx"] == torch.tensor([11, 3], device="cuda")).all()
        c.check(out)


def test_ties_go_to_the_lowest_index():
    c = Case(4, 256, 128, 40, 0, 5, True)
    c.inputs["router"][:] = c.inputs["router"][7].clone()
    out = c.run()
    assert (out["idx"] == torch.arange(5, device="cuda")).all()
    c.inputs["x"].zero_()
    out = c.run()
    assert (out["idx"] == torch.arange(5, device="cuda")).all()
    assert (out["output"] == 0).all() and torch.allclose(out["weights"], torch.full_like(out["weights"], 0.2))


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_and_unreached_weights_stay_by_themselves(fp8, bad):
    c = Case(9, 256, 144, 32, 1, 2, fp8)
    good = c.run()
    used = set(good["idx"].flatten().tolist()) | {0, 1, 32}
    for j in range(33):
        if j not in used:
            if fp8:
                c.inputs["gate_up"][j].view(torch.uint8).fill_(0x7f)
                c.inputs["down_scales"][j] = float("nan")
            else:
                c.inputs["gate_up"][j] = float("nan")
                c.inputs["down"][j] = float("nan")
    again = c.run()
    for name in good:
        assert torch.equal(good[name], again[name])
    c.inputs["x"][4, 100] = bad
    out = c.run()
    assert not torch.isfinite(out["output"][4]).any()
    c.check(out, [t for t in range(9) if t != 4])


@pytest.mark.parametrize("fp8", [True, False])
def test_moe_repeats_its_bits_on_another_stream_and_in_a_graph(fp8):
    c = Case(7, 1024, 640, 24, 1, 4, fp8)
    first = c.run()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        outs = [c.run() for _ in range(20)]
    stream.synchronize()
    out = c.layer.empty_outputs("moe", 7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.layer.moe(c.inputs, out)
        c.layer.moe(c.inputs, out)
    out["output"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    for other in outs + [out]:
        for name in first:
            assert torch.equal(first[name], other[name])
    c.layer.check_errors()


def test_the_optional_outputs():
    c = Case(2, 256, 128, 8, 0, 2, True)
    full = c.run()
    only = c.layer.moe(c.inputs, {"output": torch.empty_like(full["output"])})
    assert torch.equal(only["output"], full["output"])


def test_moe_refusals():
    from mhc_residual_boundary_gb300 import Sublayer, capi
    for kw, text in (({"hidden": 250}, "multiples of 16"), ({"intermediate": 0}, "multiples of 16"),
                     ({"hidden": 32768}, "hidden or intermediate >"), ({"experts": 513}, "num_experts >"),
                     ({"top_k": 9}, "top_k"), ({"top_k": 0}, "top_k"), ({"shared_experts": 9}, "shared_experts"),
                     ({"max_moe_tokens": 33}, "max_moe_tokens"), ({"max_moe_tokens": 0}, "max_moe_tokens")):
        args = dict(hidden=256, intermediate=128, experts=8, top_k=2, max_moe_tokens=4)
        with pytest.raises(capi.MhcError, match=text):
            Sublayer(**{**args, **kw})
    with pytest.raises(ValueError, match="score"):
        Sublayer(score="tanh")
    c = Case(4, 256, 128, 8, 0, 2, True)
    out = c.layer.empty_outputs("moe", 4)
    five = torch.zeros(5, 256, dtype=BF16, device="cuda")
    with pytest.raises(capi.MhcError, match="MHC_ERR_CAPACITY"):
        c.layer.moe(dict(c.inputs, x=five), c.layer.empty_outputs("moe", 5))
    with pytest.raises(capi.MhcError, match="MHC_ERR_CAPACITY"):
        c.layer.moe(dict(c.inputs, x=five[:0]), c.layer.empty_outputs("moe", 0))
    with pytest.raises(ValueError, match="gate_up"):
        c.layer.moe(dict(c.inputs, gate_up=c.inputs["gate_up"][:, :128]), out)
    with pytest.raises(ValueError, match="router"):
        c.layer.moe(dict(c.inputs, router=c.inputs["router"].float()), out)
    with pytest.raises(ValueError, match="must be a tensor on"):
        c.layer.moe(dict(c.inputs, x=c.inputs["x"].cpu()), out)
    bare = Sublayer()
    with pytest.raises(capi.MhcError, match="without experts"):
        capi.mhc_sublayer_moe(bare.handle, capi.mhc_sublayer_moe_args_t())
    with pytest.raises(capi.MhcError, match="x is NULL"):
        a = capi.mhc_sublayer_moe_args_t()
        a.m = 1
        capi.mhc_sublayer_moe(c.layer.handle, a)


@pytest.mark.parametrize("fp8", [True, False])
def test_stalled_copies_report_a_timeout_and_the_handle_recovers(fp8):
    from mhc_residual_boundary_gb300 import capi
    c = Case(3, 512, 256, 8, 1, 2, fp8)
    good = c.run()
    torch.cuda.synchronize()
    capi.mhc_test_stall_sublayer_copies(True)
    try:
        c.run()
        torch.cuda.synchronize()
    finally:
        capi.mhc_test_stall_sublayer_copies(False)
    with pytest.raises(capi.MhcError, match="MHC_ERR_TIMEOUT"):
        c.layer.check_errors()
    c.layer.check_errors()
    again = c.run()
    for name in good:
        assert torch.equal(good[name], again[name])
    c.layer.check_errors()


def test_many_calls_one_after_another():
    """The shapes that keep every part of the pipeline busy, many times: the
    CTAs' order in time changes, the result may not."""
    for args in ((1, 5120, 2048, 16, 1, 8, True), (32, 1024, 1024, 32, 1, 8, True), (5, 1024, 512, 16, 0, 2, False)):
        c = Case(*args)
        first = c.run()
        out = c.layer.empty_outputs("moe", c.m)
        for _ in range(20):
            for _ in range(25):
                c.layer.moe(c.inputs, out)
            for name in first:
                assert torch.equal(first[name], out[name])
        c.layer.check_errors()


def test_the_widest_scales_of_many_tokens():
    """32 k blocks an item and 30 tokens an expert: the stages leave the scales
    no room beyond what the layout reserves after them."""
    c = Case(30, 128, 16384, 2, 0, 2, True)
    c.check(c.run())
    c.layer.check_errors()

"""The MoE layer's sigmoid scores, bit for bit: 1 / (1 + exp(-logit)) with a
correctly rounded quotient, so that scores near one order, and tie, as the
definition's do in FP32.

x is one in one place, so that an expert's logit is its router weight there.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("low,high", [(-20.0, 20.0), (3.0, 18.0), (-90.0, -60.0), (14.0, 17.0)])
@pytest.mark.parametrize("experts", [33, 200, 512])
def test_sigmoid_scores(experts, low, high):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mhc_residual_boundary_gb300 import Sublayer
    m, h, i, k = 32, 64, 16, 16
    g = torch.Generator(device="cuda").manual_seed(experts)
    layer = Sublayer(hidden=h, intermediate=i, experts=experts, top_k=k, max_moe_tokens=m, fp8=False,
                     score="sigmoid", renormalize=False, router_f32=True)
    router = low + (high - low) * torch.rand(experts, h, generator=g, device="cuda")
    x = torch.zeros(m, h, dtype=BF16, device="cuda")
    x[torch.arange(m), torch.arange(m)] = 1.0
    inp = {"x": x, "router": router, "gate_up": torch.zeros(experts, 2 * i, h, dtype=BF16, device="cuda"),
           "down": torch.zeros(experts, h, i, dtype=BF16, device="cuda")}
    for bias in (None, torch.randint(-2, 3, (experts,), generator=g, device="cuda").float() * 4):
        if bias is not None:
            inp["bias"] = bias
        out = layer.moe(inp, layer.empty_outputs("moe", m))
        score = 1.0 / (1.0 + torch.exp(-router[:, :m].t().contiguous()))
        ranked = score if bias is None else score + bias
        idx = torch.sort(ranked, dim=1, descending=True, stable=True)[1][:, :k]
        assert torch.equal(out["idx"].long(), idx)
        assert torch.equal(out["weights"], score.gather(1, idx))
    layer.check_errors()

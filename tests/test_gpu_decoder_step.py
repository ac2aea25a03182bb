"""examples/decoder_step.py: the operators together with the boundary.  Each
operator's outputs are checked against its definition in 64 bits from the
inputs that the step gave it (the tolerances are the operators' own), the MoE
layer's against a call by itself, and a captured step against a called one."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from test_gpu_sublayer import check_bf16, check_product, check_quantized, silu_product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    spec = importlib.util.spec_from_file_location("decoder_step", os.path.join(ROOT, "examples", "decoder_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("m", [1, 13, 32])
def test_step(example, m):
    s = example.DecoderStep(m, hidden=1024, tp=4, mlp=1280, intermediate=384, experts=16, shared_experts=1, top_k=4,
                            vocab=2056, seed=m)
    logits = s.step().clone()
    s.check_errors()

    def product(a, w, out):
        check_product(out["output"], {"values": a["values"], "scales": a["scales"], "weight": w[0],
                                      "weight_scales": w[1]})
    check_quantized(s.x8, s.at[0]["layer_input"].double())
    product(s.x8, s.gate_up, s.gate_up_out)
    check_quantized(s.h8, silu_product(s.gate_up_out["output"]))
    product(s.h8, s.down, s.mlp_out)
    alone = s.sub.empty_outputs("moe", m)
    s.sub.moe({"x": s.at[1]["layer_input"].clone(), "router": s.router, "bias": s.bias, **s.experts}, alone)
    for name in alone:
        assert torch.equal(alone[name], s.moe_out[name]), name
    r = s.moe_out["output"].double() + s.at[2]["layer_input"].double()
    check_bf16(s.final["residual_out"], r, "residual_out")
    y = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt()
    check_bf16(s.final["output"], y, "output")
    check_quantized(s.final, y)
    product(s.final, s.head, s.logits)
    assert torch.isfinite(logits).all()

    graph = s.capture()
    s.logits["output"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.logits["output"], logits)
    s.check_errors()


def test_the_last_sublayer_counts_once(example):
    """The head's boundary is not given the MoE layer's output, which the final
    norm adds: other experts change that output and the sum by the same, and
    nothing that it is added to."""
    def step(change):
        s = example.DecoderStep(5, hidden=1024, tp=2, mlp=640, intermediate=384, experts=8, shared_experts=1, top_k=2,
                                vocab=512, seed=3)
        if change:
            s.experts["down_scales"] *= -3.0
        s.step()
        s.check_errors()
        return s

    a, b = step(False), step(True)
    assert not torch.equal(a.moe_out["output"], b.moe_out["output"])
    for k in range(3):
        for name in a.at[k]:
            assert torch.equal(a.at[k][name], b.at[k][name]), (k, name)
    for s in (a, b):
        r = s.moe_out["output"].double() + s.at[2]["layer_input"].double()
        check_bf16(s.final["residual_out"], r, "residual_out")

"""How the MoE layer with 8-bit weights holds its BF16 activations: exactly down
to 2^-17 of a row's largest magnitude, off by at most 2^-25 of it below.

Each row has one value that is much larger than the others and meets only zero
weights, so the others carry the sums.  Tolerance: as in test_gpu_moe.py, with
that error of x (none down to 2^-17).
"""
import pytest
import torch

from test_gpu_moe import F8, STEPS, blocks, gen, randn

pytestmark = pytest.mark.gpu


def layer_inputs(g, m, h, i, experts, small, largest, random_signs):
    """Small values of [1, 2) * small, with all eight significant bits in use."""
    x = small * (1 + torch.randint(0, 128, (m, h), generator=g, device="cuda") / 128.0)
    if random_signs:
        x = x * torch.where(torch.rand(m, h, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    at = torch.randint(0, h, (1,), generator=g, device="cuda").item()
    x[:, at] = largest
    inp = {"x": x.bfloat16(), "router": (randn(g, experts, h) / h ** 0.5).bfloat16(),
           "gate_up": (100 * randn(g, experts, 2 * i, h)).clamp(-448, 448).to(F8),
           "down": (100 * randn(g, experts, h, i)).clamp(-448, 448).to(F8),
           "gate_up_scales": (0.5 + torch.rand(experts, 2, blocks(i), blocks(h), generator=g, device="cuda"))
           / (100 * h ** 0.5 * small),
           "down_scales": (0.5 + torch.rand(experts, blocks(h), blocks(i), generator=g, device="cuda"))
           / (100 * i ** 0.5)}
    assert torch.equal(inp["x"].float(), x)
    inp["router"][:, at] = 0
    inp["gate_up"].view(torch.uint8)[:, :, at] = 0
    return inp


def check(out, inp, x_error):
    """One route a token, of weight 1."""
    i = inp["down"].shape[2]

    def spread(s, rows, cols):
        return s.double().repeat_interleave(128, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    for j in range(inp["down"].shape[0]):
        token = (out["idx"][:, 0] == j).nonzero()[:, 0]
        if not len(token):
            continue
        x = inp["x"][token].double()
        h = x.shape[1]
        gate, up = inp["gate_up"][j].double().view(2, i, h)
        gate, up = (w * spread(s, i, h) for w, s in zip((gate, up), inp["gate_up_scales"][j]))
        down = inp["down"][j].double() * spread(inp["down_scales"][j], h, i)
        gv, uv = x @ gate.t(), x @ up.t()
        g_err = STEPS * (x.abs() @ gate.abs().t()) + x_error * gate.abs().sum(1)
        u_err = STEPS * (x.abs() @ up.abs().t()) + x_error * up.abs().sum(1)
        silu = gv * torch.sigmoid(gv)
        hv = silu * uv
        pad = torch.nn.functional.pad(hv.abs(), (0, blocks(i) * 128 - i)).view(len(token), -1, 128)
        top = pad.amax(2).repeat_interleave(128, 1)[:, :i]
        h_err = 1.1 * uv.abs() * g_err + silu.abs() * u_err + STEPS * hv.abs() + 2.0 ** -12 * hv.abs() + 2.0 ** -22 * top
        y = hv @ down.t()
        bound = h_err @ down.abs().t() + 2 * STEPS * (hv.abs() @ down.abs().t())
        bound = bound + torch.ldexp(torch.ones_like(y), torch.frexp(y.abs() + bound)[1] - 9)
        off = (out["output"][token].double() - y).abs()
        assert (off <= bound).all(), ((off / bound).max().item(), (off > bound).nonzero()[:4].tolist())


@pytest.mark.parametrize("m,experts", [(1, 1), (7, 1), (9, 2), (32, 3)])
@pytest.mark.parametrize("below", [8, 12, 13, 14, 15, 16, 17, 19, 23])
@pytest.mark.parametrize("size", [0, 30, -60])
def test_small_values_beside_a_large_one(m, experts, below, size):
    """Small values from 2^-below of the row's largest on."""
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mhc_residual_boundary_gb300 import Sublayer
    h, i = 272, 144
    layer = Sublayer(hidden=h, intermediate=i, experts=experts, top_k=1, max_moe_tokens=m)
    for largest, signs in ((1.0, True), (1.0, False), (1.9921875, True)):
        largest *= 2.0 ** size
        small = 2.0 ** (size - below) * (2 if largest > 2.0 ** size else 1)   # at least 2^-below of the largest
        inp = layer_inputs(gen(m + below), m, h, i, experts, small, largest, signs)
        out = layer.moe(inp, layer.empty_outputs("moe", m))
        assert torch.isfinite(out["output"]).all()
        check(out, inp, 0.0 if below <= 17 else 2.0 ** -25 * largest)
    layer.check_errors()

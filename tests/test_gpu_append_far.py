"""append's angles at far positions, at frequencies whose turns a position are many.

The angle in turns is a product of integers and off by 2^-64 * |position| <= 2^-33, of which 32 bits are
used, a signed number that FP32 rounds by 2^-24 of itself; sine and cosine are off by 2^-22 of 1: together less
than 2^-20 before the result is rounded to BF16."""
import math
from fractions import Fraction

import pytest
import torch

from attention_cases import BF16, half_ulp_bf16
from test_attention_turns_host import two_pi

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_and_large_frequencies(interleaved):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mhc_residual_boundary_gb300 import Attention
    d, t = 64, 96
    f = [1.0, 1000.0, -1000.0, 12345678.9, -2.0 ** 39 - 1.25, math.pi * 1e6, 0.3, 1e-7] * 4
    x = torch.zeros(t, 1, d, dtype=BF16, device="cuda")
    x[..., 0::2] = 1.0
    if not interleaved:
        x = torch.cat([torch.ones_like(x[..., :32]), torch.zeros_like(x[..., :32])], -1).contiguous()
    positions = torch.tensor([2 ** 31 - 1 - 22222222 * i for i in range(t - 3)] + [-2 ** 31, 1, -1], dtype=torch.int32,
                             device="cuda")
    q_out = torch.empty_like(x)
    with Attention(heads=1, kv_heads=1, head_dim=d, page_size=16, rotary_dim=d, frequencies=f, interleaved=interleaved) as a:
        cache = a.empty_cache(t // 16)
        a.append({"q": x, "k": x, "v": x, "positions": positions, "slots": torch.arange(t, device="cuda").int()},
                 {"q_out": q_out, **cache})
        a.check_errors()
    turn = [Fraction(v) / two_pi() for v in f[:8]]
    for i in range(8):
        angles = [2 * math.pi * float((int(p) * turn[i] + Fraction(1, 2)) % 1 - Fraction(1, 2)) for p in positions.tolist()]
        a0, b0 = (2 * i, 2 * i + 1) if interleaved else (i, i + 32)
        for at, fn in ((a0, math.cos), (b0, math.sin)):
            want = torch.tensor([fn(w) for w in angles], dtype=torch.float64, device="cuda")
            assert ((q_out[:, 0, at].double() - want).abs() <= half_ulp_bf16(want) + 2.0 ** -20).all(), (i, at)

"""One query over an 8-bit cache: weights far below the largest one, which together matter."""
import math

import pytest
import torch

from attention_cases import BF16, F32, I32, STEPS, define, gen, half_ulp_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def test_a_long_flat_rest_behind_a_few_large_weights():
    """One query over an 8-bit cache: each warp of a sequence has one position in front whose weight is 1, then only
    ones of 2^-25.2, with all of the output's value.

    FP16 weights reach from 2^15 down to 2^-24, with 7 bits above the reference for its growth of 2^8: those of 2^-14 of the
    reference over 2^7 and more are rounded by 2^-11 of themselves, smaller ones by 2^-25 / 2^7 of the reference, which is
    at most the largest weight, 1 / sum.  So an output is off by at most 2^-32 * n * max |v| / sum on top of
    the usual."""
    page, n, d = 128, 16384, 64
    from mhc_residual_boundary_gb300 import Attention
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    b, gap = 2 * sms, 25.2 * math.log(2)   # as many sequences as CTAs: each has one
    k = torch.zeros(n // page, 1, page, d, device="cuda")
    v = (0.5 + torch.rand(n // page, 1, page, d, generator=gen(9), device="cuda")) * 256
    k.view(n, d)[0:128:32, 0] = 256.0
    v.view(n, d)[0:128:32] = 0.0
    scales = torch.full((n // page, 1, page), 2.0 ** -8, dtype=F32, device="cuda")
    q = torch.zeros(b, 1, d, dtype=BF16, device="cuda")
    q[..., 0] = 16.0
    table = torch.arange(n // page, dtype=I32, device="cuda").expand(b, -1).contiguous()   # all read the same pages
    inputs = {"q": q, "k_cache": k.to(torch.float8_e4m3fn), "v_cache": v.to(torch.float8_e4m3fn), "k_scales": scales,
              "v_scales": scales.clone(), "pages": table, "lengths": torch.full((b,), n, dtype=I32, device="cuda")}
    first = {**inputs, "q": q[:1], "pages": table[:1], "lengths": inputs["lengths"][:1]}
    out, lse, mag, size = define(first, page=page, scale=gap / 16)
    with Attention(heads=1, kv_heads=1, head_dim=d, page_size=page, fp8=True) as a:
        got = a.attend(inputs, a.empty_outputs(b), scale=gap / 16)
        a.check_errors()
    before = (2.0 ** -11 + 2 * (size + 2)[..., None] * STEPS) * mag + 2.0 ** -32 * n * 1.5 / 4
    limit = half_ulp_bf16(out.abs() + before) + before
    assert ((out / limit).amin() > 50).all()
    bad = ~((got["output"].double() - out).abs() <= limit)
    assert not bad.any(), (int(bad.sum()), got["output"][0, 0, :4].tolist(), out[0, 0, :4].tolist())
    assert ((got["lse"].double() - lse).abs() <= (size + lse.abs() + 2) * STEPS).all()

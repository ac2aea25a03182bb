"""attend over values near their type's largest, and over small ones, with the tolerances of tests/attention_cases.py."""
import pytest
import torch

from attention_cases import BF16, check, define, gen, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def call(inputs, page, **kw):
    from mhc_residual_boundary_gb300 import Attention
    heads, d = inputs["q"].shape[1:]
    with Attention(heads=heads, kv_heads=inputs["k_cache"].shape[1], head_dim=d, page_size=page,
                   fp8="k_scales" in inputs) as a:
        out = a.attend(inputs, a.empty_outputs(inputs["q"].shape[0]), **kw)
        a.check_errors()
    return out


@pytest.mark.parametrize("lengths", [[1], [300, 17], [9000]])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("several", [False, True])
def test_large_values(several, fp8, d, lengths):
    """Values up to the type's largest: their weighted means are finite, though the sum of two is not.  With scores
    that grow along the sequence, so that the largest weight comes last."""
    queries = [min(n, 40) for n in lengths] if several else None
    inputs = make_inputs(3, lengths=lengths, queries=queries, heads=8, kv=2, d=d, page=64, fp8=fp8)
    largest = float(torch.finfo(BF16).max)
    if fp8:
        inputs["v_scales"] *= 0.99 * largest / 448 / inputs["v_scales"].amax()
    else:
        v = inputs["v_cache"]
        share = torch.rand(v.shape, generator=gen(4), device="cuda")
        v.copy_((0.5 + 0.5 * share) * largest)
        v[:, :, ::3] *= -1
        v[:, :, :, 5] = largest
    inputs["q"][..., 0] = 1.0
    at = torch.zeros(inputs["k_cache"].shape[0], 64, device="cuda")
    for s, n in enumerate(lengths):
        for i in range(-(-n // 64)):
            at[inputs["pages"][s, i]] = (i * 64 + torch.arange(64, device="cuda")) / n
    # scores from 0 to 12 beside the random ones: the reference of the exponentials lags behind
    k = inputs["k_cache"].float()
    k[..., 0] = at[:, None] * 12 * d ** 0.5 / (inputs["k_scales"] if fp8 else 1.0)
    inputs["k_cache"] = k.clamp(-448, 448).to(inputs["k_cache"].dtype) if fp8 else k.to(BF16)
    want = define(inputs, page=64)
    assert torch.isfinite(want[0].to(BF16)).all()
    got = call(inputs, 64)
    assert torch.isfinite(got["output"]).all()
    check(got, inputs, page=64, want=want)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("several", [False, True])
def test_small_values(several, fp8):
    """Small values keep their bits.  A position's part of a sum is off by 2^-112 (BF16 cache) at most, or by
    2^-126 * 448 * 2^20 (8 bits): over 300 positions 2^-18 of a value of 2^-86 and more, of 2^-70 and more."""
    inputs = make_inputs(5, lengths=[300, 1], queries=[40, 1] if several else None, heads=8, kv=2, d=128, page=64, fp8=fp8)
    if fp8:
        inputs["v_scales"] *= 2.0 ** -66
    else:
        inputs["v_cache"] = (inputs["v_cache"].float() * 2.0 ** -84).to(BF16)
    check(call(inputs, 64), inputs, page=64)

"""Queries that see nothing."""
import math

import pytest
import torch

from attention_cases import check, define, make_inputs

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


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_queries_that_see_nothing_hold_anything(fp8, d, value):
    """Queries before their sequence's first position, in one tile with ones that see something, and queries over pages
    that are not there: zeros and minus infinity, whatever the query holds."""
    from mhc_residual_boundary_gb300 import Attention, capi
    page = 32
    inputs = make_inputs(13, lengths=[20, 0, 70], queries=[33, 4, 3], heads=8, kv=2, d=d, page=page, fp8=fp8)
    want = define(inputs, page=page)
    inputs["q"][:13] = value
    inputs["q"][33:37] = value
    got = call(inputs, page)
    check(got, inputs, page=page, want=want)
    assert (got["output"][:13] == 0).all() and (got["lse"][:13] == -math.inf).all()
    assert (got["output"][33:37] == 0).all() and (got["lse"][33:37] == -math.inf).all()
    # no page of sequence 2 is there
    inputs["pages"][2] = -1
    inputs["q"][37:] = value
    with Attention(heads=8, kv_heads=2, head_dim=d, page_size=page, fp8=fp8) as a:
        got = a.attend(inputs, a.empty_outputs(40))
        with pytest.raises(capi.MhcError, match="INVALID_ARG"):
            a.check_errors()
    assert (got["output"][37:] == 0).all() and (got["lse"][37:] == -math.inf).all()
    assert torch.isfinite(got["output"]).all()


@pytest.mark.parametrize("several", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_minus_infinity_only(several, d):
    """Rows whose scores are all minus infinity are as rows that see nothing; a finite score beside such ones is all
    that counts."""
    inputs = make_inputs(17, lengths=[1, 130, 200], queries=[1, 1, 1] if several else None, heads=8, kv=2, d=d, page=16,
                         fp8=False)
    inputs["q"][..., 0] = 1.0
    inputs["k_cache"][..., 0] = -math.inf
    at = int(inputs["pages"][2, 150 // 16]), 1, 150 % 16
    inputs["k_cache"][at[0], at[1], at[2], 0] = 0.5
    got = call(inputs, 16)
    none = torch.ones(3, 8, dtype=torch.bool, device="cuda")
    none[2, 4:] = False
    assert (got["output"][none] == 0).all() and (got["lse"][none] == -math.inf).all()
    value = inputs["v_cache"][at].expand(4, d)
    assert torch.equal(got["output"][2, 4:], value) and torch.isfinite(got["lse"][2, 4:]).all()

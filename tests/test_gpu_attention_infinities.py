"""One query a sequence: infinities and NaN among the values that it sees, as the definition has them.

An infinity times a weight is an infinity of its sign, so a column with infinities of one sign is infinite, one with
both signs, or a NaN, is NaN; the other columns are those of the finite values, within the tolerances of
tests/attention_cases.py.  (No weight here is so small that it vanishes in FP32: scores differ by less than 60.)
"""
import math

import pytest
import torch

from attention_cases import check, define, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def place(inputs, spots, page):
    for s, position, head, column, value in spots:
        inputs["v_cache"][int(inputs["pages"][s, position // page]), head, position % page, column] = value


def compare(inputs, page, **kw):
    from mhc_residual_boundary_gb300 import Attention
    heads, d = inputs["q"].shape[1:]
    out, lse, mag, size = define(inputs, page=page, **kw)
    with Attention(heads=heads, kv_heads=inputs["k_cache"].shape[1], head_dim=d, page_size=page) as a:
        got = a.attend(inputs, a.empty_outputs(inputs["q"].shape[0]), **kw)
        a.check_errors()
    assert torch.isinf(out).any() and torch.isnan(out).any()
    assert torch.equal(torch.isnan(got["output"]), torch.isnan(out))
    infinite = torch.isinf(out)
    assert torch.equal(torch.isinf(got["output"]), infinite)
    assert torch.equal(got["output"][infinite].double(), out[infinite])
    fine = torch.isfinite(out)
    got["output"] = torch.where(fine, got["output"], 0.0)
    check(got, inputs, page=page, want=(torch.where(fine, out, 0.0), lse, torch.where(fine, mag, 0.0), size))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 8, 16])
def test_one_position(d, group):
    """Its weight is 1, whatever the score."""
    inputs = make_inputs(3, lengths=[1, 1, 1], heads=2 * group, kv=2, d=d, page=16, fp8=False)
    place(inputs, [(0, 0, 0, 3, math.inf), (0, 0, 1, d - 1, -math.inf), (1, 0, 1, 0, math.nan), (2, 0, 0, 1, -math.inf)], 16)
    compare(inputs, 16)


@pytest.mark.parametrize("window, sinks", [(0, 0), (60, 5)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 12])
def test_some_positions(d, group, window, sinks):
    page, lengths = 16, [300, 47, 1, 260, 129]
    inputs = make_inputs(5, lengths=lengths, heads=2 * group, kv=2, d=d, page=page, fp8=False)
    spots = [(0, 299, 0, 3, math.inf), (0, 290, 0, 3, math.inf), (0, 288, 1, 7, -math.inf), (0, 1, 1, 5, math.inf),
             (0, 2, 1, 5, -math.inf), (0, 295, 0, d - 1, math.nan), (1, 46, 1, 33, -math.inf), (1, 0, 1, 34, math.inf),
             (3, 100, 0, 2, math.inf), (3, 259, 0, 9, math.inf), (3, 250, 0, 9, -math.inf), (4, 128, 1, 63, -math.inf),
             (4, 127, 1, 62, math.inf), (4, 126, 1, 62, math.inf), (4, 125, 0, 0, math.nan)]
    place(inputs, spots, page)
    compare(inputs, page, window=window, sinks=sinks)


def test_every_position_and_every_part():
    """A long sequence that many CTAs have parts of: one column is infinite everywhere, one in one place."""
    page = 64
    inputs = make_inputs(7, lengths=[30011], heads=8, kv=1, d=128, page=page, fp8=False)
    inputs["v_cache"][..., 17] = -math.inf
    place(inputs, [(0, 12345, 0, 2, math.inf), (0, 0, 0, 100, math.inf), (0, 30010, 0, 101, -math.inf),
                   (0, 20000, 0, 55, math.nan)], page)
    compare(inputs, page)

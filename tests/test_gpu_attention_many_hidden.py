"""More queries before their sequence's first position than 2^31 pieces of 16 bytes of output: all of their rows are
written.  (69 GB of queries and output.)"""
import math

import pytest
import torch

from attention_cases import BF16, F32, I32, check, make_inputs

pytestmark = pytest.mark.gpu


def test_queries_that_see_nothing_fill_more_than_2_31_pieces():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mhc_residual_boundary_gb300 import Attention
    heads, d, page, t, n = 8, 128, 64, 2 ** 24, 5
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("needs 100 GB of free memory")
    assert t * heads * d // 8 >= 2 ** 31
    inputs = make_inputs(3, lengths=[n], queries=[n], heads=heads, kv=heads, d=d, page=page, fp8=False)
    q = torch.empty(t, heads, d, dtype=BF16, device="cuda")
    q[-n:] = inputs["q"]
    out = {"output": torch.full((t, heads, d), 3.0, dtype=BF16, device="cuda"),
           "lse": torch.full((t, heads), 3.0, dtype=F32, device="cuda")}
    with Attention(heads=heads, kv_heads=heads, head_dim=d, page_size=page) as a:
        a.attend({**inputs, "q": q, "q_starts": torch.tensor([0, t], dtype=I32, device="cuda")}, out)
        a.check_errors()
    step = 2 ** 19
    for i in range(0, t - step, step):
        assert not out["output"][i:i + step].any(), i
    assert not out["output"][t - step:-n].any() and (out["lse"][:-n] == -math.inf).all()
    check({name: x[-n:] for name, x in out.items()}, inputs, page=page)
    del q, out
    torch.cuda.empty_cache()

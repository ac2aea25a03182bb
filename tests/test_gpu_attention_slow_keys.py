"""Values that arrive before the keys: the cache's values are in the L2, its keys are not, nor are the keys of another
call's cache.  A part of the cache that has not arrived must not be taken for one that has."""
import pytest
import torch

from attention_cases import check, define, make_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slow", ["k_cache", "v_cache"])
@pytest.mark.parametrize("heads, kv, d, fp8, lengths, queries", [
    (32, 4, 128, False, [6000, 5000, 3001, 6000, 900, 6000, 4500, 257], [4] * 8),
    (64, 2, 128, False, [3000] * 12, None),
    (8, 2, 128, False, [4000, 4096], [600, 1024]),
    (32, 4, 64, False, [6000, 5000, 3001, 6000], [4] * 4),
    (32, 4, 128, True, [6000, 5000, 3001, 6000, 900], [4] * 5),
    (32, 4, 128, False, [6000, 5000, 3001, 6000, 900], None),
])
def test_one_side_of_the_cache_is_far(heads, kv, d, fp8, lengths, queries, slow):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mhc_residual_boundary_gb300 import Attention
    inputs = make_inputs(3, lengths=lengths, queries=queries, heads=heads, kv=kv, d=d, page=64, fp8=fp8)
    fast = inputs["v_cache" if slow == "k_cache" else "k_cache"].view(torch.uint8)
    flush = torch.empty(512 * 2 ** 20, dtype=torch.uint8, device="cuda")   # four times the L2
    want = define(inputs, page=64)
    with Attention(heads=heads, kv_heads=kv, head_dim=d, page_size=64, fp8=fp8) as a:
        first = a.attend(inputs, a.empty_outputs(inputs["q"].shape[0]))
        a.check_errors()
        check(first, inputs, page=64, want=want)
        out = a.empty_outputs(inputs["q"].shape[0])
        for i in range(40):
            flush.fill_(i)
            fast.max()
            a.attend(inputs, out)
            assert all(torch.equal(out[n], first[n]) for n in out), i
        a.check_errors()

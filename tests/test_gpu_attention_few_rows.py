"""Calls whose tiles have few rows over long caches, again and again: most of a tile's warps are done before the one
with the rows, which has to be waited for before the kernel gives its tensor memory back."""
import random

import pytest
import torch

from attention_cases import check, make_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads, kv, d, fp8, sequences, queries, length", [
    (32, 4, 128, False, 8, 4, 20000),    # proposed tokens
    (32, 4, 128, True, 8, 3, 9000),
    (20, 1, 64, False, 100, 1, 5000),
    (128, 4, 128, False, 64, 1, 8192),   # one query of more than 16 heads for each kv head
    (64, 2, 128, True, 33, 1, 6000),
])
def test_few_rows_many_times(heads, kv, d, fp8, sequences, queries, length):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mhc_residual_boundary_gb300 import Attention
    rng = random.Random(heads + length)
    lengths = [length] + [rng.randint(1, length) for _ in range(sequences - 1)]
    if queries == 1:
        lengths[3] = lengths[-1] = 0
    inputs = make_inputs(3, lengths=lengths, queries=None if queries == 1 and heads // kv > 16 else [queries] * sequences,
                         heads=heads, kv=kv, d=d, page=64, fp8=fp8)
    with Attention(heads=heads, kv_heads=kv, head_dim=d, page_size=64, fp8=fp8) as a:
        first = a.attend(inputs, a.empty_outputs(inputs["q"].shape[0]))
        a.check_errors()
        check(first, inputs, page=64)
        outs = [a.empty_outputs(inputs["q"].shape[0]) for _ in range(4)]
        for i in range(400):
            a.attend(inputs, outs[i % 4])
        a.check_errors()
        for out in outs:
            assert all(torch.equal(out[n], first[n]) for n in out)
